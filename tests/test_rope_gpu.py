"""qk_norm_rope and its gradients against the 64-bit reference, element by element within bounds
that follow from the kernels' arithmetic (paged_reference.py)."""
import numpy as np
import pytest
import torch

import tiled_attention_10_gb300 as fa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def np64(t):
    return t.detach().double().cpu().numpy()


def bshd(t, layout):
    a = np64(t)
    return a.transpose(0, 2, 1, 3) if layout == "BNSD" else a


def make(B, S, H, H_kv, D, rot, axes, layout, dtype, seed, views=False, pos_lo=0, pos_hi=5000):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def rows(h):
        shape = (B, h, S, D) if layout == "BNSD" else (B, S, h, D)
        return torch.randn(shape, generator=g).to(dt)

    if views:      # views of one fused projection
        x = rows(H + 2 * H_kv).cuda()
        q, k = (x[:, :H], x[:, H:H + H_kv]) if layout == "BNSD" else (x[:, :, :H], x[:, :, H:H + H_kv])
    else:
        q, k = rows(H).cuda(), rows(H_kv).cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda() for _ in range(2)]
    pos = torch.randint(pos_lo, pos_hi, (axes, B, S), generator=g).to(torch.int32).cuda()
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).cuda() if rot else None
    axis = [int(i) for i in torch.randint(0, axes, (rot // 2,), generator=g)] if axes > 1 else None
    d = [torch.randn(t.shape, generator=g).to(dt).cuda() for t in (q, k)]
    return q, k, w, pos, freq, axis, d


CASES = [
    # B, S, H, H_kv, D, rot, axes, layout, dtype, views
    (1, 1, 1, 1, 64, 64, 1, "BSND", "bf16", False), (1, 1, 32, 8, 128, 128, 1, "BSND", "bf16", True),
    (2, 37, 4, 2, 128, 128, 3, "BNSD", "bf16", False), (1, 257, 3, 1, 64, 32, 1, "BSND", "f16", True),
    (3, 19, 5, 5, 128, 16, 2, "BNSD", "f16", True), (2, 130, 28, 4, 128, 96, 4, "BSND", "bf16", False),
    (1, 700, 8, 2, 64, 48, 3, "BSND", "bf16", True), (2, 5, 64, 8, 128, 0, 1, "BSND", "f16", False),
    (1, 3000, 2, 2, 128, 128, 1, "BNSD", "f16", False), (4, 1, 7, 1, 64, 64, 2, "BNSD", "bf16", False),
    (1, 5000, 16, 4, 64, 64, 1, "BSND", "bf16", False),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward_and_gradients(cuda_lib, c, norm, interleaved):
    B, S, H, H_kv, D, rot, axes, layout, dtype, views = c
    if not norm and not rot:
        pytest.skip("nothing to do: refused (see the host tests)")
    q, k, w, pos, freq, axis, d = make(*c[:9], seed=S + H, views=views)
    if not norm:
        w = [None, None]
    kw = dict(q_weight=w[0], k_weight=w[1], norm=norm, eps=EPS, pair_axis=axis, interleaved=interleaved, layout=layout)
    got = fa.qk_norm_rope(q, k, pos if rot else None, freq, **kw)
    grads = fa.qk_norm_rope_backward(d[0], d[1], q, k, pos if rot else None, freq, **kw)
    ang = ref.angles(pos.cpu().numpy(), freq.cpu().numpy(), axis) if rot else np.zeros((B, S, 1, 0))
    for i, x in enumerate((q, k)):
        wx = None if w[i] is None else np64(w[i])
        x64, d64 = bshd(x, layout), bshd(d[i], layout)
        y = ref.norm_rope(x64, wx, ang, norm, EPS, interleaved)
        b = ref.norm_rope_bound(x64, wx, ang, norm, EPS, interleaved, x.dtype)
        assert (np.abs(bshd(got[i], layout) - y) <= b).all()
        dx, dw = ref.norm_rope_grad(d64, x64, wx, ang, norm, EPS, interleaved)
        bx, bw = ref.norm_rope_grad_bounds(d64, x64, wx, ang, norm, EPS, interleaved, x.dtype)
        assert (np.abs(bshd(grads[i], layout) - dx) <= bx).all()
        if norm:
            assert (np.abs(np64(grads[2 + i]) - dw) <= bw).all()
        else:
            assert grads[2 + i] is None


@pytest.mark.parametrize("lo,hi", [(-(2 ** 31), -(2 ** 31) + 50), (2 ** 31 - 50, 2 ** 31 - 1), (-5, 5), (2 ** 20, 2 ** 21)])
def test_far_and_negative_positions(cuda_lib, lo, hi):
    q, k, w, pos, freq, axis, _ = make(1, 40, 2, 1, 64, 64, 1, "BSND", "f16", 3, pos_lo=lo, pos_hi=hi)
    got = fa.qk_norm_rope(q, k, pos, freq, norm=False, layout="BSND")
    ang = ref.angles(pos.cpu().numpy(), freq.cpu().numpy(), None)
    for x, y in zip((q, k), got):
        b = ref.norm_rope_bound(np64(x), None, ang, False, EPS, False, x.dtype)
        assert (np.abs(np64(y) - ref.norm_rope(np64(x), None, ang, False, EPS, False)) <= b).all()


def test_odd_frequencies(cuda_lib):
    q, k, w, pos, freq, axis, _ = make(1, 33, 2, 1, 64, 16, 1, "BSND", "bf16", 4)
    freq = torch.tensor([0.0, -1.0, 7.0, 100.5, float("inf"), float("nan"), -float("inf"), 1e-12], dtype=torch.float64).cuda()
    got = fa.qk_norm_rope(q, k, pos, freq, layout="BSND")
    used = torch.where(torch.isfinite(freq), freq, torch.zeros_like(freq))
    ang = ref.angles(pos.cpu().numpy(), used.cpu().numpy(), None)
    b = ref.norm_rope_bound(np64(q), None, ang, True, EPS, False, q.dtype)
    assert (np.abs(np64(got[0]) - ref.norm_rope(np64(q), None, ang, True, EPS, False)) <= b).all()


def test_values_at_the_ends_of_the_type(cuda_lib):
    """All zeros (the norm of nothing), denormals, the largest values, and a NaN that stays in its row."""
    q = torch.zeros(1, 6, 2, 64, dtype=torch.float16, device="cuda")
    q[0, 1] = 6e-8
    q[0, 2] = 65504.0
    q[0, 3] = torch.linspace(-1, 1, 64, device="cuda").half()
    q[0, 4] = q[0, 3]
    q[0, 4, 1, 5] = float("nan")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    got, _ = fa.qk_norm_rope(q, q.clone(), pos, freq, eps=EPS, layout="BSND")
    ang = ref.angles(pos.cpu().numpy().reshape(1, 1, 6), freq.cpu().numpy(), None)
    want = ref.norm_rope(np64(q), None, ang, True, EPS, False)
    ok = np.ones((6, 2), bool)
    ok[4, 1] = False
    b = ref.norm_rope_bound(np64(q), None, ang, True, EPS, False, q.dtype)
    assert (np.abs(np64(got) - want) <= b)[0][ok].all()
    assert torch.isnan(got[0, 4, 1]).all()
    dq, _, dw, _ = fa.qk_norm_rope_backward(q[:, :4].contiguous(), q[:, :4].contiguous(), q[:, :4].contiguous() * 0,
                                            q[:, :4].contiguous() * 0, pos[:4], freq, q_weight=torch.ones_like(q[0, 0, 0]),
                                            eps=0.5, layout="BSND")
    assert torch.isfinite(dq).logical_or(q[:, :4].abs() > 6e4).all() and (dw == 0).all()


def test_in_place_and_views_as_outputs(cuda_lib):
    q, k, w, pos, freq, axis, _ = make(2, 50, 4, 2, 128, 128, 1, "BSND", "bf16", 5, views=True)
    want = fa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1], layout="BSND")
    buf = torch.full((2, 50, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1], layout="BSND", out=(buf[:, :, :4], buf[:, :, 4:6]))
    assert torch.equal(buf[:, :, :4], want[0]) and torch.equal(buf[:, :, 4:6], want[1]) and (buf[:, :, 6:] == 7).all()
    v_before = q._base[:, :, 6:].clone()
    fa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1], layout="BSND", out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(q._base[:, :, 6:], v_before)


def test_packed_tokens_and_positions_shapes(cuda_lib):
    q, k, w, pos, freq, axis, _ = make(1, 60, 4, 2, 64, 64, 1, "BSND", "bf16", 6)
    want = fa.qk_norm_rope(q, k, pos, freq, layout="BSND")
    for p in (pos, pos[0], pos[0, 0]):
        got = fa.qk_norm_rope(q, k, p, freq, layout="BSND")
        assert torch.equal(got[0], want[0])
    for p in (pos[0], pos[0, 0]):
        got = fa.qk_norm_rope(q[0], k[0], p, freq)
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1][0])
    two = torch.cat((q, q)), torch.cat((k, k))
    got = fa.qk_norm_rope(*two, pos[0, 0], freq, layout="BSND")
    assert torch.equal(got[0][1], want[0][0])
    empty = fa.qk_norm_rope(q[0, :0], k[0, :0], pos[0, 0, :0], freq)
    assert empty[0].shape == (0, 4, 64)
    _, _, dw, _ = fa.qk_norm_rope_backward(q[0, :0], k[0, :0], q[0, :0], k[0, :0], pos[0, 0, :0], freq, q_weight=w[0])
    assert (dw == 0).all()
    for bad in (pos.long(), pos[0, 0, :-1], pos.expand(2, 1, 60)[:, :, :-1], None):
        with pytest.raises((TypeError, ValueError)):
            fa.qk_norm_rope(q, k, bad, freq, layout="BSND")


def test_autograd_matches_the_backward_call(cuda_lib):
    q, k, w, pos, freq, axis, d = make(2, 33, 4, 2, 64, 64, 2, "BNSD", "bf16", 7)
    leaves = [t.clone().requires_grad_() for t in (q, k, *w)]
    kw = dict(pair_axis=axis, interleaved=True)
    out = fa.qk_norm_rope(leaves[0], leaves[1], pos, freq, q_weight=leaves[2], k_weight=leaves[3], **kw)
    got = torch.autograd.grad(out, leaves, d)
    want = fa.qk_norm_rope_backward(d[0], d[1], q, k, pos, freq, q_weight=w[0], k_weight=w[1], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # an expanded gradient, an output without a gradient, and frozen weights
    out = fa.qk_norm_rope(leaves[0], leaves[1], pos, freq, q_weight=w[0], k_weight=None, **kw)
    (gq,) = torch.autograd.grad(out[0].sum(), leaves[:1])
    one = torch.ones_like(q), torch.zeros_like(k)
    want = fa.qk_norm_rope_backward(*one, q, k, pos, freq, q_weight=w[0], **kw)
    assert torch.equal(gq, want[0])
    with pytest.raises(ValueError):
        fa.qk_norm_rope(leaves[0], leaves[1], pos, freq, out=(q, k), **kw)


def test_gradient_against_differences(cuda_lib):
    """The kernel's gradient against central differences of the 64-bit forward at the same inputs:
    off by the kernel's own bound along the direction, and the differences' e^2 term."""
    q, k, w, pos, freq, axis, d = make(1, 9, 2, 1, 64, 64, 1, "BSND", "f16", 8)
    grads = fa.qk_norm_rope_backward(d[0], d[1], q, k, pos, freq, q_weight=w[0], k_weight=w[1], eps=EPS, layout="BSND")
    ang = ref.angles(pos.cpu().numpy(), freq.cpu().numpy(), None)
    x, dy, wx = np64(q), np64(d[0]), np64(w[0])
    v = np.random.default_rng(2).standard_normal(x.shape)
    e = 1e-5
    diff = ((ref.norm_rope(x + e * v, wx, ang, True, EPS, False) - ref.norm_rope(x - e * v, wx, ang, True, EPS, False)) * dy).sum() / (2 * e)
    bx, _ = ref.norm_rope_grad_bounds(dy, x, wx, ang, True, EPS, False, q.dtype)
    assert abs(diff - (np64(grads[0]) * v).sum()) <= (bx * np.abs(v)).sum() + 1e-6 * np.abs(dy * v).sum()


def test_deterministic_and_on_a_side_stream(cuda_lib):
    q, k, w, pos, freq, axis, d = make(1, 3000, 8, 2, 128, 128, 1, "BSND", "bf16", 9)
    kw = dict(q_weight=w[0], k_weight=w[1], layout="BSND")
    want = fa.qk_norm_rope_backward(d[0], d[1], q, k, pos, freq, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [fa.qk_norm_rope_backward(d[0], d[1], q, k, pos, freq, **kw) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for r in got for a, b in zip(want, r))


def test_captured_training_step(cuda_lib):
    """Norm, rotation and attention, forward and backward, captured and replayed on new inputs."""
    q, k, w, pos, freq, axis, d = make(1, 200, 4, 2, 64, 64, 1, "BNSD", "bf16", 10)
    v = torch.randn_like(k)

    def step(leaves):
        a, b = fa.qk_norm_rope(leaves[0], leaves[1], pos, freq, q_weight=leaves[3], k_weight=leaves[4])
        return torch.autograd.grad(fa.flash_attention(a, b, leaves[2], causal=True), leaves, d[0])

    static = [t.clone().requires_grad_() for t in (q, k, v, *w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static)
    with torch.no_grad():
        for t in static[:3]:
            t.mul_(0.5)
    graph.replay()
    got = [t.clone() for t in got]
    want = step([t.detach().clone().requires_grad_() for t in static])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (128, 32), (128, 112)])
def test_what_is_not_rotated_passes_unchanged(cuda_lib, D, rot, interleaved):
    """Infinities, NaN and negative zeros among the elements behind the rotation, both ways (a
    NaN's payload apart)."""
    q, k, _, pos, freq, _, _ = make(1, 21, 3, 2, D, rot, 1, "BSND", "bf16", 11)
    for x in (q, k):
        rest = x[..., rot:]
        rest[:, ::2, :, ::3] = float("inf")
        rest[:, ::3, :, 1::4] = -float("inf")
        rest[:, 1::4, :, 2::5] = float("nan")
        rest[:, 1::2, :, ::2] = -0.0
    kw = dict(norm=False, interleaved=interleaved, layout="BSND")
    for got in (fa.qk_norm_rope(q, k, pos, freq, **kw), fa.qk_norm_rope_backward(q, k, q, k, pos, freq, **kw)[:2]):
        for x, y in zip((q, k), got):
            a, b = (t[..., rot:].contiguous() for t in (x, y))
            assert torch.equal(a.isnan(), b.isnan())
            assert torch.equal(a.view(torch.int16)[~a.isnan()], b.view(torch.int16)[~a.isnan()])
            assert torch.isfinite(y[..., :rot]).all()


def test_writing_over_a_saved_tensor_is_noticed(cuda_lib):
    """Outputs written into tensors that autograd has saved: their backward says so."""
    q, k, w, pos, freq, axis, _ = make(1, 20, 4, 2, 64, 64, 1, "BSND", "bf16", 12)
    one = lambda t: torch.ones_like(t).requires_grad_()
    y, z = q * one(q), k * one(k)
    fa.qk_norm_rope(q, k, pos, freq, layout="BSND", out=(q, k))
    for t in (y, z):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            t.sum().backward()

    lens = torch.full((2,), 10, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    sl = fa.paged_slots(lens, lens, lens, table, page_size=16, total_q=20)
    y, _ = fa.qk_norm_rope(q.clone().requires_grad_(), k, sl.positions, freq, layout="BSND")
    fa.paged_slots(lens + 3, lens, lens, table, page_size=16, total_q=20, out=sl)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()

    cache = fa.KV4Cache.allocate(4, 16, 2, 64)
    slots = torch.arange(20, device="cuda")
    got = fa.kv4_read(cache, slots)
    y = [t * one(t) for t in got]
    fa.kv4_read(cache, slots, out=got)
    p = q[0].clone()
    cu, used = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"), lens
    o, lse = fa.paged_attention_kv4(p, cache, cu, used, table, max_seqlen_q=10)
    y += [o * one(o), lse * one(lse)]
    fa.paged_attention_kv4(p, cache, cu, used, table, max_seqlen_q=10, out=o, lse=lse)
    for t in y:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            t.sum().backward()


def test_a_million_heads(cuda_lib):
    """The most heads a call takes, of one token: what they are as heads of many tokens at its position."""
    n, g = 1 << 20, torch.Generator(device="cuda").manual_seed(13)
    x = [torch.randn(1, 1, n, 128, generator=g, device="cuda").bfloat16() for _ in range(4)]
    freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).cuda()
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    many = [t.view(1, 2048, n // 2048, 128) for t in x]
    for a, b in ((fa.qk_norm_rope(*x[:2], pos, freq, layout="BSND"), fa.qk_norm_rope(*many[:2], pos.expand(2048), freq, layout="BSND")),
                 (fa.qk_norm_rope_backward(*x, pos, freq, layout="BSND")[:2],
                  fa.qk_norm_rope_backward(*many, pos.expand(2048), freq, layout="BSND")[:2])):
        for y, z in zip(a, b):
            assert torch.isfinite(y).all() and torch.equal(y.view(-1), z.reshape(-1))


def test_frequencies_from_2_to_the_64_on_read_as_zero(cuda_lib):
    q, k, _, pos, _, _, _ = make(1, 20, 2, 1, 64, 16, 1, "BSND", "f16", 14, pos_lo=1)
    big = torch.tensor([2.0 ** 64, -2.0 ** 64, 1.7 * 2.0 ** 64, 2.0 ** 65, 1e300, -1e300, float("inf"), 2.0 ** 64 * (1 + 2.0 ** -52)],
                       dtype=torch.float64, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(fa.qk_norm_rope(q, k, pos, big, norm=False, layout="BSND"), (q, k)))
    below = torch.nextafter(big[0], big[0] * 0).expand(8).contiguous()
    assert not torch.equal(fa.qk_norm_rope(q, k, pos, below, norm=False, layout="BSND")[0], q)


def test_strides_past_32_bits(cuda_lib):
    """Rows of q and k, and of the outputs, more than 2^32 elements apart, both ways."""
    q, k, w, pos, freq, axis, d = make(1, 3, 2, 2, 64, 64, 1, "BSND", "bf16", 15)
    step = (1 << 32) + 64
    buf = torch.empty(2 * step + (1 << 20), dtype=torch.bfloat16, device="cuda")
    far = [buf.as_strided((1, 3, 2, 64), (8, step, 512, 1), 4096 * i) for i in range(4)]
    for a, b in zip(far, (q, k, *d)):
        a.copy_(b)
    kw = dict(q_weight=w[0], k_weight=w[1], layout="BSND")
    want, grads = fa.qk_norm_rope(q, k, pos, freq, **kw), fa.qk_norm_rope_backward(*d, q, k, pos, freq, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, fa.qk_norm_rope_backward(far[2], far[3], far[0], far[1], pos, freq, **kw)))
    fa.qk_norm_rope(far[0], far[1], pos, freq, out=(far[2], far[3]), **kw)
    assert torch.equal(far[2], want[0]) and torch.equal(far[3], want[1])
