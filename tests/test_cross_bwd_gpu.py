"""The backward of cross attention on the GPU: against the formula's gradients in 64 bits and
against differences, through autograd, in both backward modes, strided, masked and captured."""
import pytest
import torch

import _kv_ref as ref
from test_kv_gpu import DEV, NAN, i32, randn

pytestmark = pytest.mark.gpu

CASES = [  # B, Lq, Lk, lens, hq, hkv, d
    (1, 1, 1, [1], 1, 1, 64),
    (2, 5, 9, None, 4, 2, 64),
    (3, 130, 77, [77, 0, 40], 4, 4, 64),
    (2, 129, 300, [300, 131], 2, 1, 128),
    (2, 257, 128, [127, 128], 6, 2, 128),
    (3, 64, 520, [1, 513, 256], 7, 1, 64),
    (1, 300, 385, None, 2, 2, 128),
    (2, 40, 641, [600, 384], 8, 2, 128),
]


def inputs(case, seed):
    B, Lq, Lk, lens, hq, hkv, d = CASES[case]
    q, do = randn(B, Lq, hq, d, seed=seed), randn(B, Lq, hq, d, seed=seed + 1)
    kv = randn(B, Lk, 2, hkv, d, seed=seed + 2)
    for b, n in enumerate(lens or []):
        kv[b, n:] = NAN  # states past a row's count may hold anything
    return q, kv, do, lens


@pytest.fixture
def deterministic(ra_lib):
    ra_lib.ra_set_bwd_deterministic(True)
    yield
    ra_lib.ra_set_bwd_deterministic(False)


def run(ra, q, kv, do, lens, dtype):
    dev = kv.to(DEV)
    k, v = dev[:, :, 0], dev[:, :, 1]
    ln = i32(lens).to(DEV) if lens else None
    o, l = ra.cross_attn_fwd(q.to(DEV), k, v, ln, out_dtype=torch.bfloat16)
    g = ra.cross_attn_bwd(q.to(DEV), k, v, o, l, do.to(DEV), ln, grad_dtype=dtype)
    assert ra.ra_sync_status() == 0
    return g


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(ra_lib, case, dtype):
    q, kv, do, lens = inputs(case, 40 * case)
    g = run(ra_lib, q, kv, do, lens, dtype)
    want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], lens or [kv.shape[1]] * len(q), do,
                              q.shape[-1] ** -0.5)
    ref.check_grads(g, want, f"case {case}")
    for b, n in enumerate(lens or []):
        assert (g[1][b, n:] == 0).all() and (g[2][b, n:] == 0).all()


@pytest.mark.parametrize("case", range(len(CASES)))
def test_gradients_deterministic(ra_lib, deterministic, case):
    q, kv, do, lens = inputs(case, 40 * case)
    g = run(ra_lib, q, kv, do, lens, torch.float32)
    want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], lens or [kv.shape[1]] * len(q), do,
                              q.shape[-1] ** -0.5)
    ref.check_grads(g, want, f"case {case}")
    again = run(ra_lib, q, kv, do, lens, torch.float32)
    assert all(torch.equal(a, b) for a, b in zip(g, again))


@pytest.mark.parametrize("mode", [False, True])
@pytest.mark.parametrize("at", [0, 2])
def test_key_counts_out_of_bounds(ra_lib, mode, at):
    """A key count past the states is cut to them and reported, as by the forward; a negative one
    is none."""
    q, kv, do, lens = inputs(2, 17)
    kv = kv.nan_to_num(0)
    dev, lens = kv.to(DEV), list(lens)
    lens[at], lens[1] = 78, -2
    full = [77 if n > 77 else max(n, 0) for n in lens]
    o, l = ra_lib.cross_attn_fwd(q.to(DEV), dev[:, :, 0], dev[:, :, 1], i32(full).to(DEV),
                                 out_dtype=torch.bfloat16)
    assert ra_lib.ra_sync_status() == 0
    ra_lib.ra_set_bwd_deterministic(mode)
    try:
        g = ra_lib.cross_attn_bwd(q.to(DEV), dev[:, :, 0], dev[:, :, 1], o, l, do.to(DEV),
                                  i32(lens).to(DEV))
    finally:
        ra_lib.ra_set_bwd_deterministic(False)
    assert ra_lib.ra_sync_status() == 5 and ra_lib.ra_sync_status() == 0
    ref.check_grads(g, ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], full, do, 0.125), "cut")


def test_against_differences(ra_lib):
    """The gradients' inner product with a direction against the 64-bit loss's central
    difference along it (step 1e-5: its own error is about 1e-10 of the loss)."""
    q, kv, do, lens = inputs(3, 7)
    kv = kv.nan_to_num(0)
    g = run(ra_lib, q, kv, do, lens, torch.float32)
    x = [q.double(), kv[:, :, 0].double(), kv[:, :, 1].double()]
    _, bounds = ref.cross_backward(*x, lens, do, 128 ** -0.5)
    for i in range(3):
        step = torch.randn(x[i].shape, generator=torch.Generator().manual_seed(i),
                           dtype=torch.float64)

        def loss(h):
            y = list(x)
            y[i] = x[i] + h * step
            return (ref.cross_attention(*y, lens, 128 ** -0.5)[0] * do.double()).sum()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = (g[i].double().cpu() * step).sum()
        tol = (bounds[i] * step.abs()).sum() + 1e-5 * want.abs()
        assert (got - want).abs() <= tol, i


@pytest.mark.parametrize("case", [2, 3, 7])
def test_through_autograd(ra_lib, case):
    """q as a leaf, k and v as slices of one leaf: their gradients meet in it; a gradient of
    the output that arrives expanded (from a sum) is taken too."""
    from sequence_parallelism_attn_b200 import autograd
    q, kv, do, lens = inputs(case, 90)
    kv = kv.nan_to_num(0)
    ql, kvl = q.to(DEV).requires_grad_(), kv.to(DEV).requires_grad_()
    ln = i32(lens).to(DEV) if lens else None
    o = autograd.cross_attention(ql, kvl[:, :, 0], kvl[:, :, 1], ln)
    (o * do.to(DEV)).sum().backward()
    want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], lens or [kv.shape[1]] * len(q), do,
                              q.shape[-1] ** -0.5)
    ref.check_grads((ql.grad, kvl.grad[:, :, 0], kvl.grad[:, :, 1]), want)
    o = autograd.cross_attention(ql, kvl[:, :, 0], kvl[:, :, 1], ln)
    g = torch.autograd.grad(o.sum(), ql)[0]
    ones = torch.ones_like(do)
    want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], lens or [kv.shape[1]] * len(q), ones,
                              q.shape[-1] ** -0.5)
    ref.check_grads((g,), ([want[0][0]], [want[1][0]]))


def test_captured_step(ra_lib):
    """Forward and backward captured together; key counts change between replays."""
    q, kv, do, lens = inputs(2, 11)
    kv = kv.nan_to_num(0)
    qd, kd, dd = q.to(DEV), kv.to(DEV), do.to(DEV)
    ln = i32(lens).to(DEV)

    def step():
        o, l = ra_lib.cross_attn_fwd(qd, kd[:, :, 0], kd[:, :, 1], ln, out_dtype=torch.bfloat16)
        return ra_lib.cross_attn_bwd(qd, kd[:, :, 0], kd[:, :, 1], o, l, dd, ln)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step()
    for now in ([77, 0, 40], [3, 77, 64]):
        ln.copy_(i32(now))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], now, do, 0.125)
        ref.check_grads(g, want, str(now))


@pytest.mark.parametrize("B,Lq", [(0, 5), (2, 0)])
def test_no_queries(ra_lib, B, Lq):
    """Without a query the results are empty and k's and v's gradients zero."""
    from sequence_parallelism_attn_b200 import autograd
    q, k, v = (torch.ones(B, n, h, 64, device=DEV).bfloat16().requires_grad_()
               for n, h in ((Lq, 4), (7, 2), (7, 2)))
    o = autograd.cross_attention(q, k, v)
    assert o.shape == (B, Lq, 4, 64) and o.dtype == torch.bfloat16
    g = torch.autograd.grad(o, (q, k, v), torch.zeros_like(o))
    assert [x.shape for x in g] == [x.shape for x in (q, k, v)] and not any(x.any() for x in g)
    assert ra_lib.cross_attn_fwd(q, k, v)[1].shape == (B, 4, Lq)
    assert ra_lib.ra_sync_status() == 0


def test_fp32_inputs_are_refused(ra_lib):
    from sequence_parallelism_attn_b200 import autograd
    x = torch.zeros(1, 2, 2, 64, device=DEV)
    with pytest.raises(ValueError):
        autograd.cross_attention(x, x, x)
    with pytest.raises(ValueError):
        ra_lib.cross_attn_bwd(x.bfloat16(), x.bfloat16(), x.bfloat16(), x, x[..., 0], x)


def test_captured_training_step(ra_lib):
    """A training step through autograd, captured: the gradients of every replay are those of
    the inputs that it finds."""
    from sequence_parallelism_attn_b200 import autograd
    q, kv, do, lens = inputs(7, 21)
    kv = kv.nan_to_num(0)
    ql, kl, vl = (x.to(DEV).contiguous().requires_grad_()
                  for x in (q, kv[:, :, 0], kv[:, :, 1]))
    dd, ln = do.to(DEV), i32(lens).to(DEV)

    def step():
        return torch.autograd.grad(autograd.cross_attention(ql, kl, vl, ln), (ql, kl, vl), dd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step()
    for seed in (22, 23):
        q = randn(*q.shape, seed=seed)
        with torch.no_grad():
            ql.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.cross_backward(q, kv[:, :, 0], kv[:, :, 1], lens, do, q.shape[-1] ** -0.5)
        ref.check_grads(g, want, str(seed))


def test_second_derivative_is_refused(ra_lib):
    """With create_graph the gradients are the same; differentiating them raises."""
    from sequence_parallelism_attn_b200 import autograd
    q, kv, do, _ = inputs(1, 31)
    x = [t.to(DEV).contiguous().requires_grad_() for t in (q, kv[:, :, 0], kv[:, :, 1])]
    plain = torch.autograd.grad(autograd.cross_attention(*x), x, do.to(DEV))
    again = torch.autograd.grad(autograd.cross_attention(*x), x, do.to(DEV), create_graph=True)
    # (one key tile: an element of dq is a single addition to zero)
    assert all(torch.equal(a, b) for a, b in zip(plain, again))
    assert not any(a.requires_grad for a in plain) and all(b.requires_grad for b in again)
    with pytest.raises((ValueError, RuntimeError), match="differentiated once"):
        torch.autograd.grad(sum(g.float().sum() for g in again) + (x[0] ** 2).sum(), x)
