"""GPU parity of the norm with rotation and its gradients against the fp64 oracle.

Tolerances, taken before the first run (u = 2^-24): 1/rms is off by at most
(D/2 + 4) u relative (a sum of D squares in fp32, its square root, the
hardware's reciprocal square root at two steps), each product adds u, so a
rotated value by (D/2 + 10) u (|y_a| + |y_b|), and bf16 rounding by 2^-8 of
the value.  dx: g, w g and the mean of D products behave alike: (D + 20) u r
(|w g| + |xh| mean |w g xh| + |g pair|), and 2^-8 |dx|.  dw: each term by (D/2 + 10) u
and the sum in the order of the kernel by at most (terms per thread + 200) u
of the sum of |g xh|; with at most 200 terms per thread, (D/2 + 410) u.
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    assert torch.cuda.is_available()
    yield
    assert mcs.mcs_device_status() == 0


def _f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, B, N, Hq, Hkv, D, rot, interleaved, layout, fused, given, weights, eps=1e-6):
        g = torch.Generator(device="cuda").manual_seed(B * N + Hq + rot)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.B, self.N, self.H, self.D, self.rot, self.eps = B, N, (Hq, Hkv), D, rot, eps
        self.inter, self.layout = interleaved, layout
        stride = (Hq + 2 * Hkv) * D if fused else 0
        x = (rand(B, N, (Hq + 2 * Hkv) * D) * 3).to(BF)
        x[:, -1] = 0  # a row of zeros: 1/sqrt(eps)
        self.buf = x
        self.q = x[..., :Hq * D].view(B, N, Hq, D)
        self.k = x[..., Hq * D:(Hq + Hkv) * D].view(B, N, Hkv, D)
        if not fused:
            self.q, self.k = self.q.contiguous(), self.k.contiguous()
        self.w = [1 + 0.3 * rand(D) if weights else None for _ in range(2)]
        rows = N + 5
        angle = rand(rows, rot // 2).double() * 3
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.pos = torch.randint(0, rows, (B, N), generator=g, device="cuda", dtype=torch.int32) if given else None
        self.dy = [rand(*self.out_shape(h)).to(BF) for h in self.H]
        self.p = mcs.rope_params(B, N, Hq, Hkv, D, rot, rows, interleaved, layout, eps, stride, stride)
        self.fused = fused

    def out_shape(self, h):
        return (self.B, self.N, h, self.D) if self.layout == mcs.LAYOUT_BNHD else (self.B, h, self.N, self.D)

    def token_major(self, t):
        a = _f64(t)
        return a if self.layout == mcs.LAYOUT_BNHD else a.transpose(0, 2, 1, 3)

    def positions(self):
        return np.broadcast_to(np.arange(self.N), (self.B, self.N)) if self.pos is None else self.pos.cpu().numpy()

    def args(self):
        return (self.q, self.k, *self.w, self.cos, self.sin, self.pos)

    def oracle(self, i):
        w = np.ones(self.D) if self.w[i] is None else _f64(self.w[i])
        return (_f64((self.q, self.k)[i]), w, _f64(self.cos), _f64(self.sin), self.positions(), self.rot,
                self.inter, self.eps)

    def forward(self):
        outs = [torch.full(self.out_shape(h), 9.0, dtype=BF, device="cuda") for h in self.H]
        mcs.mcs_qk_norm_rope(self.p, *self.args(), *outs)
        return outs

    def backward(self, weights=True):
        B, N, D, (Hq, Hkv) = self.B, self.N, self.D, self.H
        if self.fused:
            buf = torch.full_like(self.buf, 9.0)
            dx = [buf[..., :Hq * D].view(B, N, Hq, D), buf[..., Hq * D:(Hq + Hkv) * D].view(B, N, Hkv, D)]
        else:
            buf, dx = None, [torch.full((B, N, h, D), 9.0, dtype=BF, device="cuda") for h in self.H]
        dw = [torch.full((D,), 9.0, device="cuda") if weights else None for _ in range(2)]
        ws = mcs.empty_workspace(mcs.mcs_qk_norm_rope_backward_workspace(self.p))
        mcs.mcs_qk_norm_rope_backward(self.p, *self.dy, *self.args(), *dx, *dw, ws)
        if self.fused:
            assert (buf[..., (Hq + Hkv) * D:] == 9).all()  # v's part stays
        return dx, dw


def _mix(y, rot, interleaved):
    """|y_a| + |y_b| of each value's pair."""
    z = np.abs(y)
    a, b = po._pairs(y.shape[-1], rot, interleaved)
    z[..., a], z[..., b] = z[..., a] + z[..., b], z[..., a] + z[..., b]
    return z


CASES = [  # B, N, Hq, Hkv, D, rot, interleaved, layout, fused, given, weights
    (1, 1, 1, 1, 128, 128, True, 0, False, False, True), (1, 1, 1, 0, 64, 64, False, 1, False, False, True),
    (2, 9, 8, 2, 128, 128, False, 0, True, True, True), (3, 7, 5, 3, 64, 32, True, 1, True, False, True),
    (1, 33, 12, 12, 128, 64, False, 0, False, True, False), (2, 17, 9, 1, 64, 16, False, 0, True, False, True),
    (1, 50, 40, 8, 128, 0, False, 1, True, False, True), (64, 1, 32, 8, 128, 96, False, 1, True, True, True),
    (1, 1000, 3, 2, 128, 112, True, 0, False, False, True), (1, 129, 16, 16, 64, 48, False, 1, False, True, False)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(int(x)) for x in c))
def test_forward_matches_oracle(case):
    c = Case(*case)
    for i, got in enumerate(c.forward()):
        if c.H[i] == 0:
            continue
        x, w, *rest = c.oracle(i)
        want = po.norm_rope(x, w, *rest)
        tol = 2.0 ** -8 * np.abs(want) + (c.D / 2 + 10) * U * _mix(want, c.rot, c.inter) * 2 ** 0.5
        assert (np.abs(c.token_major(got) - want) <= tol).all()
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(int(x)) for x in c))
def test_backward_matches_oracle(case):
    c = Case(*case)
    dx, dw = c.backward()
    for i in range(2):
        if c.H[i] == 0:
            assert (dw[i] == 9).all()
            continue
        x, w, *rest = c.oracle(i)
        dy = c.token_major(c.dy[i])
        want, want_w, size = po.norm_rope_backward(dy, x, w, *rest)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + c.eps)
        g = _mix(dy, c.rot, c.inter) * np.abs(w)
        xh = np.abs(x * r)
        tol = 2.0 ** -8 * np.abs(want) + (c.D + 20) * U * r * (g + xh * (g * xh).mean(-1, keepdims=True))
        assert (np.abs(_f64(dx[i]) - want) <= tol).all()
        gx = (_mix(dy, c.rot, c.inter) * xh).sum((0, 1, 2))
        assert (np.abs(_f64(dw[i]) - want_w) <= (c.D / 2 + 410) * U * gx).all()
    # without the weights' gradients the same dx
    again, _ = c.backward(weights=False)
    assert all(torch.equal(a, b) for a, b in zip(dx, again))


@pytest.mark.parametrize("case", [
    (2, 5003, 2, 1, 64, 64, False, 0, True, True, True), (1, 9801, 20, 1, 128, 32, True, 1, False, False, True),
    (3, 3301, 1, 0, 128, 128, False, 1, False, True, False), (1, 10007, 3, 4, 64, 48, True, 0, False, True, True),
    (1, 9999, 1, 12, 128, 128, True, 0, True, True, True),
    # and many of more heads: blocks that take several units, two and four rows per thread
    (1, 4999, 8, 16, 128, 96, False, 0, True, True, True), (2, 1501, 40, 10, 128, 128, True, 1, False, True, True),
    (1, 6007, 16, 9, 64, 64, False, 1, False, True, True)], ids=lambda c: "-".join(str(int(x)) for x in c))
def test_many_tokens_of_few_heads(case):
    """Warps that take several tokens (one, both or no tensors of such a call), with padding among them."""
    c = Case(*case)
    skip = torch.zeros(c.B, c.N, dtype=torch.bool, device="cuda")
    if c.pos is not None:
        skip = torch.rand(c.B, c.N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.2
        c.pos[skip] = -1
    live = ~skip.cpu().numpy()
    outs, (dx, dw) = c.forward(), c.backward()
    assert mcs.mcs_device_status() == 0
    for i in range(2):
        if c.H[i] == 0:
            continue
        x, w, cos, sin, pos, *rest = c.oracle(i)
        pos = np.maximum(pos, 0)
        want = po.norm_rope(x, w, cos, sin, pos, *rest)
        tol = 2.0 ** -8 * np.abs(want) + (c.D / 2 + 10) * U * _mix(want, c.rot, c.inter) * 2 ** 0.5
        got = c.token_major(outs[i])
        assert (np.abs(got - want) <= tol)[live].all() and (got[~live] == 9).all()
        dy = c.token_major(c.dy[i]) * live[..., None, None]
        want, want_w, _ = po.norm_rope_backward(dy, x, w, cos, sin, pos, *rest)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + c.eps)
        g, xh = _mix(dy, c.rot, c.inter), np.abs(x * r)
        tol = 2.0 ** -8 * np.abs(want) + (c.D + 20) * U * r * (g * np.abs(w) + xh * (g * np.abs(w) * xh).mean(-1, keepdims=True))
        got = _f64(dx[i])
        assert (np.abs(got - want) <= tol)[live].all() and (got[~live] == 9).all()
        assert (np.abs(_f64(dw[i]) - want_w) <= (c.D / 2 + 410) * U * (g * xh).sum((0, 1, 2))).all()


def test_gradients_match_differences_of_the_kernel():
    """dx . e against (f(x + h e) - f(x - h e)) / 2h of the kernel's own forward pass, f = y . dy.
    bf16 outputs round by 2^-8 of each value, so f is off by about sqrt(n) 2^-9 |y dy|; a step of
    2^-2 of x keeps the quotient's error near 2 % of |e| |dx|, and the bound is five times that."""
    c = Case(1, 64, 4, 4, 128, 128, True, 0, False, False, True)
    dx, _ = c.backward()
    x0 = c.q.clone()
    g = torch.Generator(device="cuda").manual_seed(0)
    e = dx[0].float() / dx[0].float().norm() * x0.float().norm()  # along the gradient
    e[:, -1] = 0
    h = 2.0 ** -4
    vals, xs = [], []
    for s in (1, -1):
        c.q = (x0.float() + s * h * e).to(BF)
        xs.append(c.q.double())
        y = c.forward()[0].double()
        vals.append(float((y * c.dy[0].double()).sum()))
    moved = (xs[0] - xs[1])  # the step that was really taken
    want = float((moved * dx[0].double()).sum())
    # second-order terms cancel; the third order is h^2 of the first at most
    assert abs(vals[0] - vals[1] - want) <= 0.1 * abs(want)


def test_in_place_and_padding_positions():
    c = Case(2, 12, 4, 2, 128, 64, False, mcs.LAYOUT_BNHD, False, True, True)
    want = c.forward()
    q, k = c.q.clone(), c.k.clone()
    mcs.mcs_qk_norm_rope(c.p, q, k, *c.w, c.cos, c.sin, c.pos, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # padding tokens (and positions past the table) keep their rows and add nothing
    dx0, dw0 = c.backward()
    skip = torch.zeros(2, 12, dtype=torch.bool, device="cuda")
    skip[0, 3] = skip[1, 11] = skip[1, 0] = True
    c.pos[skip] = -1
    got = c.forward()
    dx, dw = c.backward()
    assert mcs.mcs_device_status() == 0
    for a, b in zip(got + dx, want + dx0):
        assert (a[skip] == 9).all() and torch.equal(a[~skip], b[~skip])
    for i in range(2):
        x, w, cos, sin, pos, *rest = c.oracle(i)
        dy = c.token_major(c.dy[i]) * ~skip.cpu().numpy()[..., None, None]
        _, want_w, _ = po.norm_rope_backward(dy, x, w, cos, sin, np.maximum(pos, 0), *rest)
        size = (_mix(dy, c.rot, c.inter) * np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + c.eps)).sum((0, 1, 2))
        assert (np.abs(_f64(dw[i]) - want_w) <= (c.D / 2 + 410) * U * size).all()
    c.pos[skip] = c.p.table_rows
    got = c.forward()
    assert mcs.mcs_device_status() == 6
    assert all((a[skip] == 9).all() for a in got)
    # dq in dq_out's place
    c.pos[skip] = 0
    dx0, _ = c.backward()
    ws = mcs.empty_workspace(mcs.mcs_qk_norm_rope_backward_workspace(c.p))
    mcs.mcs_qk_norm_rope_backward(c.p, *c.dy, *c.args(), *c.dy, None, None, ws)
    assert torch.equal(c.dy[0], dx0[0]) and torch.equal(c.dy[1], dx0[1])


def test_layouts_agree_and_feed_the_attention():
    """The BHND and BNHD outputs hold the same bits, and go into mcs_dense_attn as they are."""
    outs = []
    for layout in (mcs.LAYOUT_BHND, mcs.LAYOUT_BNHD):
        c = Case(1, 300, 4, 4, 128, 128, True, layout, True, False, True)
        q, k = c.forward()
        p = mcs.params(1, 4, 300, 128, layout=layout)
        out = torch.empty_like(q)
        mcs.mcs_dense_attn(p, q, k, q, out)
        outs.append([t if layout == mcs.LAYOUT_BHND else t.transpose(1, 2) for t in (q, k, out)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_weight_gradients_repeat_bit_for_bit_also_in_a_graph():
    c = Case(1, 3001, 12, 4, 128, 128, True, 0, True, False, True)
    (dx, dw), (dx2, dw2) = c.backward(), c.backward()
    assert all(torch.equal(a, b) for a, b in zip(dx + dw, dx2 + dw2))
    ws = mcs.empty_workspace(mcs.mcs_qk_norm_rope_backward_workspace(c.p))
    outs = [torch.zeros_like(t) for t in dw]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mcs.mcs_qk_norm_rope_backward(c.p, *c.dy, *c.args(), *dx2, *outs, ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, dw))


@pytest.mark.parametrize("case", [
    # heads that do not fill a warp's 4, 8 or 16, two and four rows per thread
    (1, 9, 5, 3, 128, 128, True, 0, False, False, True), (2, 17, 9, 1, 64, 16, False, 0, True, False, True),
    (1, 50, 40, 10, 128, 64, False, 1, True, True, True), (1, 2500, 9, 10, 128, 0, False, 1, False, True, True),
    # several tokens per warp, with rows left over
    (2, 5003, 2, 1, 64, 64, False, 0, True, True, True), (1, 9999, 1, 12, 128, 128, True, 0, True, True, True),
    (3, 3301, 1, 0, 128, 128, False, 1, False, True, False), (1, 10007, 3, 4, 64, 48, True, 0, False, False, True)],
    ids=lambda c: "-".join(str(int(x)) for x in c))
def test_gradients_without_eps(case):
    """eps = 0 and no row of zeros: rows that do not exist and padding add nothing to the weights'
    gradients.  Tolerances as above."""
    c = Case(*case, eps=0.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (c.q, c.k):
        t[:, -1] = torch.randn(t[:, -1].shape, generator=g, device="cuda").to(BF)
    skip = torch.zeros(c.B, c.N, dtype=torch.bool, device="cuda")
    if c.pos is not None:
        skip = torch.rand(c.B, c.N, device="cuda", generator=g) < 0.2
        c.pos[skip] = -1
    live = ~skip.cpu().numpy()
    outs, (dx, dw) = c.forward(), c.backward()
    for i in range(2):
        if c.H[i] == 0:
            continue
        x, w, cos, sin, pos, *rest = c.oracle(i)
        pos = np.maximum(pos, 0)
        want = po.norm_rope(x, w, cos, sin, pos, *rest)
        tol = 2.0 ** -8 * np.abs(want) + (c.D / 2 + 10) * U * _mix(want, c.rot, c.inter) * 2 ** 0.5
        got = c.token_major(outs[i])
        assert (np.abs(got - want) <= tol)[live].all() and (got[~live] == 9).all()
        dy = c.token_major(c.dy[i]) * live[..., None, None]
        want, want_w, _ = po.norm_rope_backward(dy, x, w, cos, sin, pos, *rest)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True))
        g_, xh = _mix(dy, c.rot, c.inter), np.abs(x * r)
        tol = 2.0 ** -8 * np.abs(want) + (c.D + 20) * U * r * (g_ * np.abs(w) + xh * (g_ * np.abs(w) * xh).mean(-1, keepdims=True))
        got = _f64(dx[i])
        assert (np.abs(got - want) <= tol)[live].all() and (got[~live] == 9).all()
        assert (np.abs(_f64(dw[i]) - want_w) <= (c.D / 2 + 410) * U * (g_ * xh).sum((0, 1, 2))).all()


@pytest.mark.parametrize("case", [(1, 4999, 8, 16, 128, 96, False, 0, True, False, True),
                                  (2, 301, 40, 8, 128, 128, True, 1, False, False, True),
                                  (1, 700, 16, 32, 64, 64, False, 1, False, False, True)],
                         ids=lambda c: "-".join(str(int(x)) for x in c))
def test_gradients_with_and_without_positions(case):
    """Positions given as each token's place are the positions without any, whichever form takes them:
    dx is the same bits, dw the same sum in another order."""
    c = Case(*case)
    dx, dw = c.backward()
    c.pos = torch.arange(c.N, device="cuda", dtype=torch.int32).expand(c.B, c.N).contiguous()
    dx2, dw2 = c.backward()
    assert all(torch.equal(a, b) for a, b in zip(dx, dx2))
    for i in range(2):
        x, w, *rest = c.oracle(i)
        dy = c.token_major(c.dy[i])
        want, want_w, _ = po.norm_rope_backward(dy, x, w, *rest)
        size = (_mix(dy, c.rot, c.inter) * np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + c.eps)).sum((0, 1, 2))
        for got in (dw[i], dw2[i]):
            assert (np.abs(_f64(got) - want_w) <= (c.D / 2 + 410) * U * size).all()
