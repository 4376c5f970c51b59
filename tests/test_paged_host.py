"""CPU tests of the operators around paged attention: every refusal (before any CUDA call; the
pointers are fake and never read) and the plain references themselves."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tiled_attention_10_gb300 import binding

P = [4096 * (i + 1) for i in range(32)]       # fake aligned pointers, 4 KB apart


# ---------------------------------------------------------------- fa_paged_slots
SLOTS = dict(past=P[0], new=P[1], free=P[2], n_free=4, table=P[3], n=2, pages=8, ps=16, total=10, cu=P[4],
             used=P[5], pos=P[6], slot=P[7], taken=P[8])


def _slots(**over):
    a = dict(SLOTS, **over)
    return binding.fa_paged_slots(a["past"], a["new"], a["free"], a["n_free"], a["table"], a["n"], a["pages"],
                                  a["ps"], a["total"], a["cu"], a["used"], a["pos"], a["slot"], a["taken"])


@pytest.mark.parametrize("over,code", [
    *[({k: None}, 1) for k in ("past", "new", "free", "table", "cu", "used", "pos", "slot", "taken")],
    (dict(n=0), 1), (dict(pages=0), 1), (dict(ps=0), 1), (dict(total=-1), 1), (dict(n_free=-1), 1),
    (dict(past=P[0] + 2), 3), (dict(slot=P[7] + 4), 3), (dict(taken=P[8] + 1), 3),
    (dict(n=16385), 2), (dict(pages=1 << 31), 2), (dict(total=(1 << 31) - 1), 2), (dict(ps=1 << 40), 2),
    (dict(used=P[0]), 1), (dict(cu=P[1] + 4), 1), (dict(table=P[2] + 8), 1), (dict(pos=P[7] + 8), 1),
])
def test_slots_refusals(built_lib, over, code):
    assert _slots(**over) == code


# ---------------------------------------------------------------- fa_qk_norm_rope
DENSE = (8 * 4 * 64, 64, 4 * 64)              # [B, S, 4, 64]
ROPE = dict(q=P[0], k=P[8], qo=P[16], ko=P[24], qw=P[5], kw=P[6], pos=P[7], freq=P[9], B=1, S=8, H=4, H_kv=4,
            D=64, rot=64, axes=1, axis=None, inter=0, norm=1, eps=1e-6, st=[DENSE] * 4, dtype="bf16")


def _rope(**over):
    a = dict(ROPE, **over)
    return binding.fa_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["qw"], a["kw"], a["pos"], a["freq"], a["B"],
                                   a["S"], a["H"], a["H_kv"], a["D"], a["rot"], a["axes"], a["axis"], a["inter"],
                                   a["norm"], a["eps"], a["st"], a["dtype"])


@pytest.mark.parametrize("over,code", [
    *[({k: None}, 1) for k in ("q", "k", "qo", "ko", "pos", "freq", "st")],
    (dict(B=-1), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(rot=80), 1), (dict(rot=-2), 1), (dict(axes=0), 1),
    (dict(axes=5), 1), (dict(axes=2, axis=[0] * 31 + [2]), 1), (dict(norm=0), 1),
    (dict(norm=0, rot=0, qw=None, kw=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=9), 1),
    (dict(D=96), 2), (dict(rot=24), 2), (dict(dtype="e4m3"), 2),
    (dict(q=P[0] + 8), 3), (dict(qo=P[16] + 2), 3), (dict(freq=P[9] + 4), 3), (dict(qw=P[5] + 1), 3),
    (dict(st=[DENSE] * 3 + [(2048, 64, 260)]), 3), (dict(st=[(0, 64, 256)] + [DENSE] * 3), 1),
    # outputs over inputs: shifted by a row, over the other input, over one another, other strides in place
    (dict(qo=P[0] + 512), 1), (dict(qo=P[8]), 1), (dict(qo=P[16], ko=P[16]), 1),
    (dict(qo=P[0], st=[DENSE, DENSE, (2048, 64, 320), DENSE]), 1),
    (dict(B=0, q=None, k=None, qo=None, ko=None), 0), (dict(S=0), 0),
])
def test_rope_refusals(built_lib, over, code):
    assert _rope(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dqo=None), 1), (dict(q=None), 1), (dict(dq=None), 1), (dict(ws=None), 1), (dict(nbytes=16), 1),
    (dict(ws=P[30] + 16), 3), (dict(norm=0, qw=None, kw=None), 1), (dict(dqw=P[1] + 1), 3), (dict(dq=P[2] + 512), 1),
    (dict(dq=P[12] + 1024), 1), (dict(st=None), 1),
])
def test_rope_bwd_refusals(built_lib, over, code):
    st, n = binding.fa_qk_norm_rope_bwd_workspace_size(64)
    assert st == 0 and n % 256 == 0
    a = dict(dqo=P[2], dko=P[4], q=P[12], k=P[14], dq=P[16], dk=P[18], qw=P[5], kw=P[6], dqw=P[20], dkw=P[21], norm=1,
             st=[DENSE] * 6, ws=P[30], nbytes=n)
    a.update(over)
    assert binding.fa_qk_norm_rope_bwd(a["dqo"], a["dko"], a["q"], a["k"], a["dq"], a["dk"], a["qw"], a["kw"], a["dqw"],
                                       a["dkw"], P[7], P[9], 1, 8, 4, 4, 64, 64, 1, None, 0, a["norm"], 1e-6, a["st"],
                                       "bf16", a["ws"], a["nbytes"]) == code


def test_rope_bwd_workspace_refusals(built_lib):
    assert binding.fa_qk_norm_rope_bwd_workspace_size(0)[0] == 1
    assert binding.fa_qk_norm_rope_bwd_workspace_size(96)[0] == 2


# ---------------------------------------------------------------- the 4-bit cache
KV = dict(k=P[0], v=P[1], slot=P[2], kc=P[3], ks=P[4], vc=P[5], vs=P[6], dk=1.0, dv=1.0, n=3, H_kv=2, D=64, ps=16,
          pages=4, dtype="f16", st=[(1, 64, 128)] * 2)


def _write(**over):
    a = dict(KV, **over)
    return binding.fa_kv4_write(a["k"], a["v"], a["slot"], a["kc"], a["ks"], a["vc"], a["vs"], a["dk"], a["dv"], a["n"],
                                a["H_kv"], a["D"], a["ps"], a["pages"], a["st"], a["dtype"])


def _read(**over):
    a = dict(KV, **over)
    return binding.fa_kv4_read(a["kc"], a["ks"], a["vc"], a["vs"], a["slot"], a["k"], a["v"], a["dk"], a["dv"], a["n"],
                               a["H_kv"], a["D"], a["ps"], a["pages"], a["dtype"])


@pytest.mark.parametrize("over,code", [
    *[({k: None}, 1) for k in ("k", "v", "slot", "kc", "ks", "vc", "vs")],
    (dict(n=-1), 1), (dict(H_kv=0), 1), (dict(pages=0), 1), (dict(ps=8), 1), (dict(dk=0.0), 1), (dict(dv=-1.0), 1),
    (dict(dk=float("nan")), 1), (dict(dv=float("inf")), 1), (dict(dk=2.0 ** -101), 1), (dict(dtype=7), 1),
    (dict(D=96), 2), (dict(dtype="e4m3"), 2), (dict(ps=48), 2), (dict(ps=1 << 17), 2), (dict(pages=1 << 31), 2),
    (dict(k=P[0] + 8), 3), (dict(kc=P[3] + 8), 3), (dict(vs=P[6] + 8), 3), (dict(slot=P[2] + 4), 3),
    (dict(n=0, k=None, v=None, slot=None), 0),
])
def test_kv4_refusals(built_lib, over, code):
    assert _write(**over) == code
    assert _read(**over) == code


@pytest.mark.parametrize("st,code", [(None, 1), ([(1, 64, 0), (1, 64, 128)], 1), ([(1, 64, 128), (1, 68, 128)], 3),
                                     ([(1, 64, 1 << 39)] * 2, 2)])
def test_kv4_write_stride_refusals(built_lib, st, code):
    assert _write(st=st) == code


ATT = dict(q=P[0], kc=P[1], ks=P[2], vc=P[3], vs=P[4], o=P[5], lse=P[6], cu=P[7], used=P[8], table=P[9], n=2, cols=8,
           ps=16, pages=20, tq=2, mq=1, tk=100, H=8, H_kv=2, D=128, scale=0.1, causal=2, dtype="bf16", dk=1.0, dv=1.0,
           ws=P[10], nbytes=1 << 40)


def _att(**over):
    a = dict(ATT, **over)
    return binding.fa_fwd_paged_kv4(a["q"], a["kc"], a["ks"], a["vc"], a["vs"], a["o"], a["lse"], a["cu"], a["used"],
                                    a["table"], a["n"], a["cols"], a["ps"], a["pages"], a["tq"], a["mq"], a["tk"], a["H"],
                                    a["H_kv"], a["D"], a["scale"], a["causal"], a["dtype"], a["dk"], a["dv"], a["ws"],
                                    a["nbytes"])


@pytest.mark.parametrize("over,code", [
    *[({k: None}, 1) for k in ("q", "kc", "ks", "vc", "vs", "o", "lse", "cu", "used", "table", "ws")],
    (dict(n=0), 1), (dict(cols=0), 1), (dict(ps=8), 1), (dict(pages=0), 1), (dict(tq=-1), 1), (dict(mq=0), 1),
    (dict(tk=-1), 1), (dict(H=7), 1), (dict(H_kv=0), 1), (dict(causal=3), 1), (dict(scale=float("inf")), 1),
    (dict(scale=3e38, dk=100.0), 1), (dict(dk=0.0), 1), (dict(dv=float("nan")), 1), (dict(dtype=5), 1), (dict(nbytes=0), 1),
    (dict(D=80), 2), (dict(dtype="e4m3"), 2), (dict(ps=48), 2), (dict(cols=1 << 28), 2), (dict(tq=1 << 31), 2),
    (dict(mq=1000, n=16385), 2),
    (dict(q=P[0] + 8), 3), (dict(ks=P[2] + 8), 3), (dict(lse=P[6] + 2), 3), (dict(ws=P[10] + 128), 3), (dict(table=P[9] + 2), 3),
    (dict(o=P[0]), 1), (dict(o=P[0] + 1024), 1),
    (dict(tq=0), 0), (dict(tq=0, q=None, o=None, lse=None), 0),
])
def test_attention_refusals(built_lib, over, code):
    assert _att(**over) == code


def test_attention_workspace(built_lib):
    size = binding.fa_fwd_paged_kv4_workspace_size
    assert size(1, 1, 100, 8, 2, 128)[0] == 0
    # decoding: partial results of the resident blocks, whatever the batch
    assert size(1, 1, 100, 8, 2, 128) == size(4000, 1, 1 << 24, 8, 2, 128)
    # long queries: 16-bit keys and values
    st, n = size(3, 4096, 10000, 8, 2, 128)
    assert st == 0 and n >= 2 * 10000 * 2 * 128 * 2
    for bad in ((0, 1, 1, 8, 2, 128), (1, 0, 1, 8, 2, 128), (1, 1, -1, 8, 2, 128), (1, 1, 1, 7, 2, 128)):
        assert size(*bad)[0] == 1
    assert size(1, 1, 1, 8, 2, 96)[0] == 2


def test_attention_workspace_serves_smaller_steps(built_lib):
    """What a step needs is never more than what one with more sequences, queries or keys is told."""
    size = lambda n, q, k, G, D: binding.fa_fwd_paged_kv4_workspace_size(n, q, k, 2 * G, 2, D)
    ns, qs, ks = (1, 7, 64, 5000), (1, 2, 5, 16, 17, 64, 128, 129, 512, 4096), (0, 100, 2047, 2048, 20000, 131071, 131072, 1 << 24)
    for G, D in ((1, 64), (4, 128), (7, 128)):
        table = {(n, q, k): size(n, q, k, G, D) for n in ns for q in qs for k in ks}
        assert all(st == 0 for st, _ in table.values())
        for (n, q, k), (_, big) in table.items():
            for a, b, c in ((n2, q2, k2) for n2 in ns for q2 in qs for k2 in ks if n2 <= n and q2 <= q and k2 <= k):
                assert table[a, b, c][1] <= big, ((a, b, c), (n, q, k))


# ---------------------------------------------------------------- torch-level checks (CPU tensors are refused)
def test_wrappers_refuse_cpu_tensors_and_wrong_types(built_lib):
    import tiled_attention_10_gb300 as fa
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_slots(i, i, i, i.view(2, 1), page_size=16, total_q=4)
    with pytest.raises(TypeError):
        fa.paged_slots(i.long(), i, i, i.view(2, 1), page_size=16, total_q=4)
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, q)
    with pytest.raises(TypeError):
        fa.qk_norm_rope(q.float(), q.float())
    with pytest.raises(ValueError):
        fa.KV4Cache.allocate(2, 16, 1, 64, device="cpu")


# ---------------------------------------------------------------- the references
def test_reference_code_rounding_is_the_nearest():
    g = np.random.default_rng(0)
    x = g.standard_normal((50, 64))
    codes, scales = ref.to_cache(x, 0.01)
    v = ref.values(codes, scales, 0.01)
    step = np.repeat(ref.e4m3_values()[scales] * float(np.float32(0.01)), 16, -1)
    grid = np.concatenate((ref.E2M1, -ref.E2M1))
    best = np.abs(x[..., None] - grid * step[..., None]).min(-1)
    assert np.allclose(np.abs(x - v), best, rtol=0, atol=1e-12)
    # the scale: no e4m3 value is nearer to amax / (6 descale)
    want = np.abs(x.reshape(50, 4, 16)).max(-1) / (6 * float(np.float32(0.01)))
    best = np.abs(want[..., None] - ref.e4m3_values()[:127]).min(-1)
    assert np.allclose(np.abs(want - ref.e4m3_values()[scales]), best, rtol=1e-12)


def test_reference_codes_match_torch_e4m3():
    b = torch.arange(256, dtype=torch.uint8)
    t = b.view(torch.float8_e4m3fn).double().numpy()
    full = np.concatenate((ref.e4m3_values(), -ref.e4m3_values()))
    assert np.array_equal(np.nan_to_num(full, nan=7777.0), np.nan_to_num(t, nan=7777.0))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_reference_gradient_against_differences(interleaved, norm):
    g = np.random.default_rng(1)
    x, dy = g.standard_normal((1, 3, 2, 64)), g.standard_normal((1, 3, 2, 64))
    w = 1 + 0.1 * g.standard_normal(64) if norm else None
    ang = g.standard_normal((1, 3, 1, 16))
    dx, dw = ref.norm_rope_grad(dy, x, w, ang, norm, 1e-3, interleaved)

    def loss(x, w):
        return (ref.norm_rope(x, w, ang, norm, 1e-3, interleaved) * dy).sum()

    e = 1e-5
    v = g.standard_normal(x.shape)
    assert abs((loss(x + e * v, w) - loss(x - e * v, w)) / (2 * e) - (dx * v).sum()) < 1e-6 * np.abs(dx * v).sum()
    if norm:
        u = g.standard_normal(64)
        assert abs((loss(x, w + e * u) - loss(x, w - e * u)) / (2 * e) - (dw * u).sum()) < 1e-6 * np.abs(dw * u).sum()


# ---------------------------------------------------------------- descales on the device
@pytest.mark.parametrize("over,code", [(dict(dk=P[20] + 2), 3), (dict(dv=P[21] + 1), 3), (dict(kc=None), 1),
                                       (dict(D=96), 2), (dict(n=0, dk=None, dv=None), 0), (dict(n=0), 0)])
def test_kv4_devscale_refusals(built_lib, over, code):
    a = dict(KV, dk=P[20], dv=P[21], **{k: v for k, v in over.items() if k not in ("dk", "dv")})
    a.update(over)
    assert binding.fa_kv4_write_devscale(a["k"], a["v"], a["slot"], a["kc"], a["ks"], a["vc"], a["vs"], a["dk"], a["dv"],
                                         a["n"], a["H_kv"], a["D"], a["ps"], a["pages"], a["st"], a["dtype"]) == code
    assert binding.fa_kv4_read_devscale(a["kc"], a["ks"], a["vc"], a["vs"], a["slot"], a["k"], a["v"], a["dk"], a["dv"],
                                        a["n"], a["H_kv"], a["D"], a["ps"], a["pages"], a["dtype"]) == code


@pytest.mark.parametrize("over,code", [(dict(dk=P[20] + 2), 3), (dict(dv=P[21] + 1), 3), (dict(scale=float("nan")), 1),
                                       (dict(D=80), 2), (dict(tq=0, dk=None, dv=None), 0), (dict(tq=0), 0)])
def test_attention_devscale_refusals(built_lib, over, code):
    a = dict(ATT, dk=P[20], dv=P[21])
    a.update(over)
    assert binding.fa_fwd_paged_kv4_devscale(
        a["q"], a["kc"], a["ks"], a["vc"], a["vs"], a["o"], a["lse"], a["cu"], a["used"], a["table"], a["n"], a["cols"],
        a["ps"], a["pages"], a["tq"], a["mq"], a["tk"], a["H"], a["H_kv"], a["D"], a["scale"], a["causal"], a["dtype"],
        a["dk"], a["dv"], a["ws"], a["nbytes"]) == code


def test_forward_mode_derivatives_are_refused():
    """A dual tensor's tangent would be dropped: refused before anything else, in every place."""
    import torch.autograd.forward_ad as fad

    import tiled_attention_10_gb300 as fa
    x, w = torch.ones(1, 2, 3, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    f = torch.ones(8, dtype=torch.float64)
    with fad.dual_level():
        dual = lambda t: fad.make_dual(t, torch.ones_like(t))
        with pytest.raises(ValueError):                # no tangent: refused as CPU tensors
            fa.qk_norm_rope(x, x)
        for q, k, kw in ((dual(x), x, {}), (x, dual(x), {}), (x, x, dict(q_weight=dual(w))), (x, x, dict(k_weight=dual(w))),
                         (x, x, dict(inv_freq=dual(f))), (dual(x.clone().requires_grad_()), x, {})):
            with pytest.raises(NotImplementedError):
                fa.qk_norm_rope(q, k, **kw)
        for args in ((dual(x), x, x, x), (x, dual(x), x, x), (x, x, dual(x), x), (x, x, x, dual(x))):
            with pytest.raises(NotImplementedError):
                fa.qk_norm_rope_backward(*args, None, None)


def test_a_gradient_of_the_frequencies_is_refused():
    import tiled_attention_10_gb300 as fa
    x = torch.ones(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.ones(8, dtype=torch.float64, requires_grad=True)
    with pytest.raises(ValueError, match="inv_freq"):
        fa.qk_norm_rope(x, x, torch.zeros(3, dtype=torch.int32), f)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(x, x, torch.zeros(3, dtype=torch.int32), f)


def test_gradients_through_the_cache_are_refused():
    """kv4_write and paged_attention_kv4 have none: refused where one is asked for, nowhere else."""
    import types

    import torch.autograd.forward_ad as fad

    import tiled_attention_10_gb300 as fa
    cache = types.SimpleNamespace(_geometry=(1, 2, 16, 64, 0))
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16)
    g = x.clone().requires_grad_()
    i = torch.zeros(1, dtype=torch.int32)
    calls = (lambda t: fa.kv4_write(t, x, None, cache), lambda t: fa.kv4_write(x, t, None, cache),
             lambda t: fa.paged_attention_kv4(t, cache, i, i, i.view(1, 1), max_seqlen_q=1))
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call(g)
        for ok in (x, g.detach()):
            with pytest.raises(ValueError, match="cuda:0"):          # only: not on a GPU
                call(ok)
        with torch.no_grad(), pytest.raises(ValueError, match="cuda:0"):
            call(g)
        with fad.dual_level(), pytest.raises(NotImplementedError):
            call(fad.make_dual(x, torch.ones_like(x)))


def test_causal_true_is_refused():
    """It would have meant top-left: a decoding query over the first key alone."""
    import types

    import tiled_attention_10_gb300 as fa
    cache = types.SimpleNamespace(_geometry=(1, 2, 16, 64, 0))
    x, i = torch.ones(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="bottom_right"):
        fa.paged_attention_kv4(x, cache, i, i, i.view(1, 1), max_seqlen_q=1, causal=True)
    for c in (False, 0, 1, 2, "none", "top_left"):
        with pytest.raises(ValueError, match="cuda:0"):
            fa.paged_attention_kv4(x, cache, i, i, i.view(1, 1), max_seqlen_q=1, causal=c)


def test_a_gradient_of_a_descale_is_refused():
    import tiled_attention_10_gb300 as fa
    cache = object.__new__(fa.KV4Cache)
    cache._geometry, cache._descales = (2, 1, 16, 64, 0), (1.0, 1.0)
    for bad in (torch.ones(1, requires_grad=True), torch.ones((), requires_grad=True)):
        with pytest.raises(ValueError, match="no gradient"):
            cache.k_descale = bad
        with pytest.raises(ValueError, match="no gradient"):
            cache.v_descale = bad
    with pytest.raises(ValueError, match="cuda:0"):                      # only: not on a GPU
        cache.k_descale = torch.ones(1)
    assert cache.k_descale == 1.0
