"""The 4-bit cache: kv4_write and kv4_read against the exact reference (codes and scales bit by
bit), and attention over it against 64-bit attention within bounds from its arithmetic."""
import itertools
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tiled_attention_10_gb300 as fa
from tests import paged_reference as ref
from tests.gpu_helpers import CANARY16, CANARY32
from tiled_attention_10_gb300 import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def np64(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def junk_cache(pages, ps, H_kv, D, kd=1.0, vd=1.0, fill=0xA5):
    c = fa.KV4Cache.allocate(pages, ps, H_kv, D, k_descale=kd, v_descale=vd)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.view(torch.uint8).fill_(fill)
    return c


def check_written(cache, k, v, slots, before):
    """Every byte of the cache: written rows by the rule, all others as before."""
    for x, codes, scales, d, old in ((k, cache.k_codes, cache.k_scales, cache.k_descale, before[0]),
                                     (v, cache.v_codes, cache.v_scales, cache.v_descale, before[1])):
        want_c, want_s = old[0].copy(), old[1].copy()
        c, s = ref.to_cache(np64(x), d)
        ps = cache.page_size
        for t, slot in enumerate(slots):
            if 0 <= slot < cache.num_pages * ps:
                want_c[slot // ps, :, slot % ps] = c[t]
                want_s[slot // ps, :, slot % ps] = s[t]
        assert np.array_equal(want_s, raw(scales))
        assert np.array_equal(want_c, raw(codes))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,H_kv,D,ps,pages", [(1, 1, 64, 16, 1), (3, 2, 128, 16, 4), (70, 8, 128, 64, 3), (257, 3, 64, 32, 20),
                                               (129, 1, 128, 128, 2), (400, 2, 64, 384, 3), (33, 5, 128, 256, 2)])
def test_write_and_read(cuda_lib, dtype, n, H_kv, D, ps, pages):
    g = torch.Generator().manual_seed(n)
    cache = junk_cache(pages, ps, H_kv, D, 0.0024, 0.7e-3)
    before = [(raw(a).copy(), raw(b).copy()) for a, b in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))]
    x = torch.randn(n, 3 * H_kv, D, generator=g).to(DT[dtype]).cuda()
    k, v = x[:, :H_kv], x[:, 2 * H_kv:]                # strided rows
    slots = torch.randperm(pages * ps, generator=g)[:n]
    slots = torch.cat((slots, torch.full((n - len(slots),), -1)))
    slots[::7] = -1
    if n > 5:
        slots[3], slots[5] = pages * ps, -(2 ** 40)     # outside: skipped
    fa.kv4_write(k, v, slots.cuda(), cache)
    check_written(cache, k, v, slots.tolist(), before)
    got = fa.kv4_read(cache, slots.cuda(), dtype=DT[dtype])
    for x, y, d, codes, scales in ((k, got[0], cache.k_descale, cache.k_codes, cache.k_scales),
                                   (v, got[1], cache.v_descale, cache.v_codes, cache.v_scales)):
        c, s = ref.to_cache(np64(x), d)
        want = ref.values(c, s, d)
        ok = ((slots >= 0) & (slots < pages * ps)).numpy()
        want[~ok] = 0.0
        # fp32 product, then one rounding
        assert (np.abs(np64(y) - want) <= ref.half_step(DT[dtype]) * 1.001 * np.abs(want) + ref.tiny(DT[dtype])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("descale", [1.0, 2.0 ** -9, 6.5 * 0.7 / 2688, 0.3, 1e-20, 1e20])
def test_borders_between_codes(cuda_lib, dtype, descale):
    """Values on, and one step beside, every border between codes and between scales."""
    dt = DT[dtype]
    d32 = float(np.float32(descale))
    rows = []
    for s in ref.e4m3_values()[[1, 2, 7, 8, 9, 15, 40, 41, 47, 86, 87, 100, 120, 126]]:
        for near in (1.0, 0.999, 1.0625, 1.0624, 1.0626):         # the group's largest: on the scale's borders too
            for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.99):
                rows.append([6 * s * d32 * near] + [b * s * d32 * (1 + j * 2.0 ** -9) * (-1) ** j for j in range(-7, 8)])
    x = torch.tensor(rows, dtype=torch.float64).to(dt)
    x = torch.cat((x, torch.zeros((-len(x)) % 4, 16, dtype=dt))).view(-1, 1, 64).cuda()
    cache = junk_cache(-(-len(x) // 16), 16, 1, 64, descale, descale)
    before = [(raw(a).copy(), raw(b).copy()) for a, b in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))]
    slots = torch.arange(len(x), device="cuda")
    fa.kv4_write(x, x.flip(0), slots, cache)
    check_written(cache, x, x.flip(0), slots.tolist(), before)


def test_every_bf16_value(cuda_lib):
    """All 65536 bit patterns, NaN and infinities among them, as elements of random groups."""
    bits = torch.randperm(65536, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).view(-1, 8, 64).cuda()
    for d in (1.0, 1e-6):
        cache = junk_cache(8, 16, 8, 64, d, d)
        before = [(raw(a).copy(), raw(b).copy()) for a, b in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))]
        fa.kv4_write(x, x, torch.arange(128, device="cuda"), cache)
        check_written(cache, x, x, list(range(128)), before)


def test_read_nan_scale_and_duplicates(cuda_lib):
    cache = junk_cache(1, 16, 1, 64, fill=0x11)
    cache.k_scales.view(torch.uint8)[0, 0, 3, 2] = 0x7F
    k, v = fa.kv4_read(cache, torch.tensor([3, 3, 99, 0], device="cuda"))
    assert torch.isnan(k[:2, 0, 32:48]).all() and torch.isfinite(k[:2, 0, :32]).all() and torch.equal(v[0], v[1])
    assert (k[2] == 0).all() and torch.isfinite(k[3]).all()


# ---------------------------------------------------------------- attention
class Step:
    """A paged step with a cache of written values, junk behind every sequence's last key."""

    def __init__(self, seq_q, seq_k, H, H_kv, D, ps, dtype, seed=0, std=1.0, kd=0.003, vd=0.002, extra_rows=0, bad_page=False):
        g = torch.Generator().manual_seed(seed)
        self.seq_q, self.seq_k, self.H, self.H_kv, self.D, self.dtype = seq_q, seq_k, H, H_kv, D, DT[dtype]
        per = [-(-n // ps) for n in seq_k]
        pages = max(1, sum(per)) + 2
        self.cache = junk_cache(pages, ps, H_kv, D, kd, vd, fill=0x7F)     # unwritten scales are NaN
        order = torch.randperm(pages, generator=g)
        cols = max(1, max(per)) + 1
        table = torch.full((len(seq_k), cols), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(per):
            table[s, :n] = order[at:at + n].int()
            at += n
        slots = [int(table[s, j // ps]) * ps + j % ps for s, n in enumerate(seq_k) for j in range(n)]
        tk = sum(seq_k)
        k = (torch.randn(tk, H_kv, D, generator=g) * std).to(self.dtype).cuda()
        v = torch.randn(tk, H_kv, D, generator=g).to(self.dtype).cuda()
        if tk:
            fa.kv4_write(k, v, torch.tensor(slots).cuda(), self.cache)
        if bad_page:
            table[0, 0] = -1
        self.table = table.cuda()
        self.used = torch.tensor(seq_k, dtype=torch.int32).cuda()
        self.cu = torch.tensor([0, *itertools.accumulate(seq_q)], dtype=torch.int32).cuda()
        self.tq = sum(seq_q) + extra_rows
        self.q = torch.randn(self.tq, H, D, generator=g).to(self.dtype).cuda()

    def run(self, causal=2, scale=None, max_q=None, **kw):
        o = torch.full((self.tq, self.H, self.D), CANARY16, dtype=torch.int16, device="cuda").view(self.dtype)
        lse = torch.full((self.H, self.tq), CANARY32, dtype=torch.int32, device="cuda").view(torch.float32)
        fa.paged_attention_kv4(self.q, self.cache, self.cu, self.used, self.table, max_seqlen_q=max_q or max(1, *self.seq_q),
                               total_k=sum(self.seq_k), scale=scale, causal=causal, out=o, lse=lse, **kw)
        return o, lse

    def check(self, o, lse, causal=2, scale=None, unpacked=None):
        scale = self.D ** -0.5 if scale is None else scale
        c = self.cache
        arrays = [(raw(a), raw(b), d) for a, b, d in ((c.k_codes, c.k_scales, c.k_descale), (c.v_codes, c.v_scales, c.v_descale))]
        table, q64, o64, l64 = self.table.cpu().numpy(), np64(self.q), np64(o), np64(lse)
        if unpacked is None:
            unpacked = max(1, *self.seq_q) * (self.H // self.H_kv) > 64
        at = 0
        for s, (nq, nk) in enumerate(zip(self.seq_q, self.seq_k)):
            k, v = (ref.gather(*a, table[s], nk, c.num_pages) for a in arrays)
            O, L, PV, A = ref.attend(q64[at:at + nq], k, v, scale, causal)
            half = ref.half_step(self.dtype)
            p_step, v_step = (half, 0.0) if unpacked else (ref.half_step(torch.float16), 0.0)
            bo, bl = ref.attend_bounds(O, PV, A, nk, self.D, self.dtype, p_step, v_step)
            rows = slice(at, at + nq)
            assert np.isfinite(o64[rows]).all()
            assert (np.abs(o64[rows] - O) <= bo).all(), (s, (np.abs(o64[rows] - O) / bo).max())
            assert np.array_equal(np.isneginf(L), np.isneginf(l64[:, rows]))
            fin = np.isfinite(L)
            assert (np.abs(l64[:, rows][fin] - L[fin]) <= bl[fin]).all()
            at += nq
        # rows of no sequence: untouched
        assert (o[at:].view(torch.int16) == CANARY16).all() and (lse[:, at:].contiguous().view(torch.int32) == CANARY32).all()


HEADS = [(1, 1), (4, 1), (8, 8), (12, 4), (28, 4), (16, 1), (8, 1), (5, 1)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_decode(cuda_lib, heads, dtype, D):
    st = Step([1, 0, 1, 1, 1, 1, 1, 0], [1, 50, 17, 300, 64, 65, 0, 0], *heads, D, 16, dtype, seed=heads[0], extra_rows=3)
    st.check(*st.run())


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256, 384])
def test_decode_page_sizes(cuda_lib, ps):
    st = Step([1] * 5, [ps - 1, ps, ps + 1, 3 * ps + 7, 1000], 8, 2, 128, ps, "bf16", seed=ps)
    st.check(*st.run())


@pytest.mark.parametrize("n", [1, 15, 16, 31, 32, 33, 63, 64, 127, 128, 129, 255, 257, 4097, 20000])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_lengths(cuda_lib, n, D):
    st = Step([1], [n], 4, 2, D, 64, "bf16", seed=n)
    st.check(*st.run())


@pytest.mark.parametrize("causal", [0, 1, 2])
@pytest.mark.parametrize("qmax,heads", [(2, (8, 2)), (4, (4, 1)), (5, (3, 1)), (8, (8, 1)), (16, (8, 2)), (64, (2, 2)), (7, (28, 4))], ids=str)
def test_several_queries(cuda_lib, qmax, heads, causal):
    st = Step([qmax, 1, 0, qmax - 1, qmax], [200, 3, 40, qmax - 1, max(1, qmax - 2)], *heads, 128, 32, "bf16", seed=qmax, extra_rows=2)
    st.check(*st.run(causal), causal)


@pytest.mark.parametrize("causal", [0, 1, 2])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("f16", 128), ("bf16", 64)])
def test_long_queries_are_unpacked(cuda_lib, dtype, D, causal):
    st = Step([130, 1, 0, 70, 300], [500, 33, 64, 20, 300], 4, 2, D, 16, dtype, seed=D, extra_rows=5)
    st.check(*st.run(causal), causal)


@pytest.mark.parametrize("causal", [0, 1, 2])
@pytest.mark.parametrize("heads,qmax,dtype,D,ps", [((8, 1), 3, "bf16", 128, 16), ((4, 2), 9, "f16", 64, 32), ((28, 4), 18, "bf16", 64, 64),
                                                   ((5, 1), 25, "f16", 128, 384), ((2, 2), 128, "bf16", 128, 64)], ids=str)
def test_17_to_128_rows(cuda_lib, heads, qmax, dtype, D, ps, causal):
    st = Step([qmax, 1, 0, qmax - 1, qmax, 2], [700, 129, 40, qmax - 2, 128, 0], *heads, D, ps, dtype, seed=qmax, extra_rows=3)
    st.check(*st.run(causal), causal, unpacked=False)


@pytest.mark.parametrize("n", [1, 63, 64, 127, 128, 129, 255, 256, 257, 4097, 20000])
def test_40_rows_over_any_length(cuda_lib, n):
    st = Step([10], [n], 8, 2, 128, 64, "bf16", seed=n)
    st.check(*st.run(), unpacked=False)


def test_more_rows_over_long_sequences(cuda_lib):
    """Several tiles of rows over sequences long enough to stay in the cache's format."""
    st = Step([128, 31, 0], [7000, 900, 5], 8, 2, 128, 64, "bf16", seed=30)
    st.check(*st.run(), unpacked=False)


@pytest.mark.parametrize("std,mul", [(30.0, 1.0), (1.0, 1e-30), (1.0, 1e30)])
def test_magnitudes_of_many_rows(cuda_lib, std, mul):
    st = Step([9, 12, 2], [700, 64, 90], 4, 1, 128, 32, "bf16", seed=5, std=std, kd=0.003 * std)
    st.q.mul_(mul)
    scale = 128 ** -0.5 / mul
    st.check(*st.run(scale=scale), scale=scale, unpacked=False)


@pytest.mark.parametrize("lens", [[30000], [513] * 40, list(range(1, 200, 3)), [128] * 300])
def test_any_split_of_many_rows(cuda_lib, lens):
    st = Step([5] * len(lens), lens, 8, 2, 64, 16, "f16", seed=8)
    o, lse = st.run()
    st.check(o, lse)
    again = st.run()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])       # deterministic


def test_both_ways_agree_at_the_border(cuda_lib):
    """The same queries through the cache as it is and, with a larger max_seqlen_q, unpacked."""
    st = Step([8, 3], [700, 90], 8, 2, 128, 64, "bf16", seed=3)
    st.check(*st.run())
    st.check(*st.run(max_q=100), unpacked=True)


@pytest.mark.parametrize("scale", [-0.08, 0.0, 1.0, 3.0])
@pytest.mark.parametrize("qn", [1, 40])
def test_scales(cuda_lib, scale, qn):
    st = Step([qn, qn], [900, 333], 4, 2, 128, 16, "bf16", seed=4)
    st.check(*st.run(scale=scale), scale=scale)


@pytest.mark.parametrize("std,mul", [(30.0, 1.0), (1.0, 1e-30), (1.0, 1e30), (1e-3, 1.0)])
def test_magnitudes(cuda_lib, std, mul):
    """Peaked and flat softmax; queries far outside f16's range, undone by the scale."""
    st = Step([1, 1, 2], [700, 64, 90], 4, 1, 128, 32, "bf16", seed=5, std=std, kd=0.003 * std)
    st.q.mul_(mul)
    scale = 128 ** -0.5 / mul
    st.check(*st.run(scale=scale), scale=scale)


def test_pages_outside_the_cache_read_as_zeros(cuda_lib):
    for qn in (1, 12, 40, 100):
        st = Step([qn, qn], [100, 70], 4, 2, 128, 16, "bf16", seed=6, bad_page=True)
        st.check(*st.run())


def test_bad_offsets_stay_inside(cuda_lib):
    """Offsets and lengths that no caller should give: nothing outside o and lse is written."""
    st = Step([1, 1, 1], [40, 50, 60], 4, 2, 64, 16, "bf16", seed=7)
    good = st.run()
    st.used[1] = -5
    st.used[2] = 2 ** 31 - 1
    st.cu.copy_(torch.tensor([0, 1, 2 ** 31 - 1, -7], dtype=torch.int32))
    o, lse = st.run()
    assert torch.equal(o[0], good[0][0])
    assert torch.isneginf(lse[:, 1]).all() and (o[1] == 0).all()


@pytest.mark.parametrize("lens", [[30000], [20000, 1, 1, 1], [513] * 40, list(range(1, 200, 3)), [64] * 700])
def test_any_split_of_the_work(cuda_lib, lens):
    st = Step([1] * len(lens), lens, 8, 4, 64, 16, "f16", seed=8)
    o, lse = st.run()
    st.check(o, lse)
    again = st.run()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])       # deterministic


def test_a_sequences_result_does_not_depend_on_rows_behind(cuda_lib):
    """The same step with a longer table, padded requests and an unordered workspace."""
    st = Step([1, 1], [300, 200], 4, 2, 128, 16, "bf16", seed=9)
    st.check(*st.run())
    ws = fa.paged_attention_kv4_workspace(st.q, st.cache, max_seqlen_q=1, n_seqs=2, total_k=500)
    ws.fill_(0xFF)
    a = st.run(workspace=ws)
    st.used = torch.cat((st.used, torch.tensor([70, 0], dtype=torch.int32, device="cuda")))
    st.cu = torch.cat((st.cu, st.cu[-1:].repeat(2)))
    st.table = torch.cat((st.table, torch.full_like(st.table, -1)))
    b = st.run(workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once(cuda_lib):
    """Calls that overlap, each with its own workspace, give what they give alone."""
    steps = [Step([1] * 40, list(range(900, 940)), 8, 2, 128, 16, "bf16", seed=20), Step([70, 9], [400, 800], 8, 2, 128, 32, "bf16", seed=21),
             Step([9] * 20, list(range(900, 920)), 8, 2, 64, 16, "bf16", seed=23)]
    alone = [st.run() for st in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[] for _ in steps]
    for _ in range(10):
        for i, (st, stream) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(stream):
                got[i].append(st.run())
    torch.cuda.synchronize()
    for a, runs in zip(alone, got):
        for b in runs:
            assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_a_wide_table_needs_no_total_k(cuda_lib):
    """More places in the block table than keys a call may count, with one query each."""
    st = Step([1, 1], [70, 130], 4, 2, 64, 64, "bf16", seed=26)
    st.check(*st.run())
    n = 4100
    table = torch.full((n, 8192), -1, dtype=torch.int32, device="cuda")
    table[:2, :st.table.shape[1]] = st.table
    used = torch.zeros(n, dtype=torch.int32, device="cuda")
    used[:2] = st.used
    cu = torch.full((n + 1,), 2, dtype=torch.int32, device="cuda")
    cu[:2] = torch.arange(2, device="cuda")
    a, b = st.run(), fa.paged_attention_kv4(st.q, st.cache, cu, used, table, max_seqlen_q=1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_workspace_for_many_steps(cuda_lib):
    """A workspace of the largest step serves steps with fewer queries and keys, whichever way they go."""
    big = Step([128] * 3, [2500, 2000, 2100], 8, 2, 64, 32, "bf16", seed=25)
    ws = fa.paged_attention_kv4_workspace(big.q, big.cache, max_seqlen_q=128, n_seqs=3, total_k=6600)
    ws.fill_(0xFF)
    big.check(*big.run(workspace=ws), unpacked=False)
    for qn in (1, 4, 9, 40, 128):
        st = Step([qn] * 3, [300, 200, 100], 8, 2, 64, 32, "bf16", seed=qn)
        st.check(*st.run(workspace=ws))


@pytest.mark.parametrize("qn", [1, 4, 9, 100])
def test_captured_over_changing_lengths(cuda_lib, qn):
    """One graph, replayed as the lengths and queries change, against calls made one by one."""
    st = Step([qn] * 3, [700, 130, 1000], 8, 2, 128, 32, "bf16", seed=24)
    ws = fa.paged_attention_kv4_workspace(st.q, st.cache, max_seqlen_q=qn, n_seqs=3, total_k=1830)
    o, lse = st.run(workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_attention_kv4(st.q, st.cache, st.cu, st.used, st.table, max_seqlen_q=qn, total_k=1830, causal=2, out=o, lse=lse, workspace=ws)
    for used in ([700, 130, 1000], [128, 129, 0], [1, 0, 999]):
        st.used.copy_(torch.tensor(used, dtype=torch.int32))
        st.q.mul_(-1.0)
        want = st.run()
        graph.replay()
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


def test_a_nan_query_stays_in_its_row(cuda_lib):
    for qn in (1, 4, 20, 80):
        st = Step([qn, qn], [300, 200], 8, 2, 128, 16, "bf16", seed=22)
        want = st.run()
        st.q[qn, 3, 7] = float("nan")
        got = st.run()
        assert torch.isnan(got[0][qn, 3]).all()
        keep = torch.ones(2 * qn, 8, dtype=torch.bool, device="cuda")
        keep[qn, 3] = False
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1].t()[keep], want[1].t()[keep])


def test_cache_past_32_bit_offsets(cuda_lib):
    """Pages whose codes and scales start beyond 2^32 bytes."""
    pages, ps = (1 << 32) // (64 * 16) + 300, 16
    pages = pages * 8 + 64                                # the scales' offsets as well: 38 GB of codes each
    c = fa.KV4Cache(*(torch.empty(pages, 1, ps, n, dtype=torch.uint8, device="cuda") for n in (64, 8, 64, 8)), 0.003, 0.003)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(50, 1, 128, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, 7, pages - 9, pages // 2 + 1]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, j // ps]) * ps + j % ps for j in range(50)]).cuda()
    fa.kv4_write(k, v, slots, c)
    rk, rv = fa.kv4_read(c, slots)
    small = fa.KV4Cache.allocate(4, ps, 1, 128, k_descale=0.003, v_descale=0.003)
    fa.kv4_write(k, v, torch.arange(50, device="cuda"), small)
    sk, sv = fa.kv4_read(small, torch.arange(50, device="cuda"))
    assert torch.equal(rk, sk) and torch.equal(rv, sv)
    used = torch.tensor([50], dtype=torch.int32, device="cuda")
    for n in (1, 4, 10, 50):
        q = torch.randn(n, 4, 128, generator=g).bfloat16().cuda()
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        a = fa.paged_attention_kv4(q, c, cu, used, table.cuda(), max_seqlen_q=n, total_k=50)
        b = fa.paged_attention_kv4(q, small, cu, used, torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4),
                                   max_seqlen_q=n, total_k=50)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_queries_and_no_tokens(cuda_lib):
    st = Step([0, 0], [20, 0], 4, 2, 64, 16, "bf16")
    o, lse = fa.paged_attention_kv4(st.q, st.cache, st.cu, st.used, st.table, max_seqlen_q=1, total_k=20)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    before = raw(st.cache.k_codes).copy()
    fa.kv4_write(none, none, slots, st.cache)
    assert np.array_equal(before, raw(st.cache.k_codes)) and fa.kv4_read(st.cache, slots)[0].shape == (0, 2, 64)


def test_wrapper_refusals(cuda_lib):
    st = Step([1], [20], 4, 2, 64, 16, "bf16")
    args = (st.q, st.cache, st.cu, st.used, st.table)
    for i, bad in ((0, st.q.float()), (0, st.q[:, :, :32].contiguous()), (2, st.cu.long()), (2, st.cu[:-1]), (3, st.used.cpu()),
                   (4, st.table.long())):
        a = list(args)
        a[i] = bad
        with pytest.raises((TypeError, ValueError)):
            fa.paged_attention_kv4(*a, max_seqlen_q=1)
    with pytest.raises(fa.FaError):
        fa.paged_attention_kv4(*args, max_seqlen_q=1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.kv4_write(st.q, st.q, torch.zeros(1, dtype=torch.int64, device="cuda"), st.cache)   # 4 heads into 2


# ---------------------------------------------------------------- the operators together
def _serve(steps, H, H_kv, D, ps, dtype, capture=False):
    """Serving steps of three requests through slots, norm and rotation, write and attention; the
    last step's outputs and everything a reference needs to redo them from the 16-bit inputs."""
    g = torch.Generator().manual_seed(11)
    n, cols = 3, 12
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(DT[dtype]).cuda() for _ in range(2)]
    cache = junk_cache(40, ps, H_kv, D, 0.003, 0.003, fill=0x7F)
    free = torch.randperm(40, generator=g).int().cuda()
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    past = torch.zeros(n, dtype=torch.int32, device="cuda")
    held = [[[], []] for _ in range(n)]
    for new in steps:
        rows = sum(new) + 2                                   # two padded rows
        x = torch.randn(rows, H + 2 * H_kv, D, generator=g).to(DT[dtype]).cuda()
        sl = fa.paged_slots(past, torch.tensor(new, dtype=torch.int32).cuda(), free, table, page_size=ps, total_q=rows)
        q, k = fa.qk_norm_rope(x[:, :H], x[:, H:H + H_kv], sl.positions, freq, q_weight=w[0], k_weight=w[1])
        fa.kv4_write(k, x[:, H + H_kv:], sl.slot_map, cache)
        o, lse = fa.paged_attention_kv4(q, cache, sl.cu_seqlens_q, sl.seqused_k, table, max_seqlen_q=max(new), total_k=400)
        at = 0
        for s, m in enumerate(new):
            held[s][0].append(np64(k[at:at + m]))
            held[s][1].append(np64(x[at:at + m, H + H_kv:]))
            at += m
        free = free[int(sl.pages_taken):]
        past = sl.seqused_k
    return q, o, lse, held, steps[-1], cache


@pytest.mark.parametrize("H,H_kv,D,ps,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "f16")])
def test_serving_steps_together(cuda_lib, H, H_kv, D, ps, dtype):
    q, o, lse, held, last, cache = _serve([[70, 5, 33], [1, 1, 1], [1, 0, 4], [1, 1, 1]], H, H_kv, D, ps, dtype)
    at = 0
    for s, nq in enumerate(last):
        kv = [ref.values(*ref.to_cache(np.concatenate(h), d), d).transpose(1, 0, 2)
              for h, d in zip(held[s], (cache.k_descale, cache.v_descale))]
        O, L, PV, A = ref.attend(np64(q[at:at + nq]), *kv, D ** -0.5, 2)
        bo, bl = ref.attend_bounds(O, PV, A, kv[0].shape[1], D, DT[dtype], ref.half_step(torch.float16), 0.0)
        assert (np.abs(np64(o[at:at + nq]) - O) <= bo).all() and (np.abs(np64(lse[:, at:at + nq]) - L) <= bl).all()
        at += nq


def test_captured_decode_step(cuda_lib):
    """One graph of the four calls, replayed over growing requests, against the calls made one by one."""
    H, H_kv, D, ps, n = 8, 2, 128, 16, 4
    g = torch.Generator().manual_seed(12)
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    x = torch.empty(n, H + 2 * H_kv, D, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    free = torch.arange(60, dtype=torch.int32, device="cuda").flip(0).contiguous()
    xs = [torch.randn(x.shape, generator=g).bfloat16().cuda() for _ in range(40)]

    def step(past, table, cache, used_pages):
        sl = fa.paged_slots(past, one, used_pages, table, page_size=ps, total_q=n)
        q, k = fa.qk_norm_rope(x[:, :H], x[:, H:H + H_kv], sl.positions, freq)
        fa.kv4_write(k, x[:, H + H_kv:], sl.slot_map, cache)
        return sl, fa.paged_attention_kv4(q, cache, sl.cu_seqlens_q, sl.seqused_k, table, max_seqlen_q=1, total_k=400)

    def fresh():
        return (torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n, 8), -1, dtype=torch.int32, device="cuda"),
                fa.KV4Cache.allocate(60, ps, H_kv, D, k_descale=0.003, v_descale=0.003))

    past, table, cache = fresh()
    pages = free.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(past, table.clone(), cache, pages)
    torch.cuda.current_stream().wait_stream(side)
    cache = fresh()[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sl, (o, lse) = step(past, table, cache, pages)
    taken, got = 0, []
    for x0 in xs:
        x.copy_(x0)
        pages[: 60 - taken].copy_(free[taken:])
        graph.replay()
        got.append((o.clone(), lse.clone()))
        taken += int(sl.pages_taken)
        past.copy_(sl.seqused_k)
    past, table, cache = fresh()
    taken = 0
    for x0, (a, b) in zip(xs, got):
        x.copy_(x0)
        sl2, (o2, l2) = step(past, table, cache, free[taken:])
        assert torch.equal(a, o2) and torch.equal(b, l2)
        taken += int(sl2.pages_taken)
        past = sl2.seqused_k


# ---------------------------------------------------------------- descales held on the device
def one(x):
    return torch.full((1,), x, dtype=torch.float32, device="cuda")


def bits(ts):
    return [t.clone().view(torch.uint8) for t in ts]


def cache_bits(c):
    return bits((c.k_codes, c.k_scales, c.v_codes, c.v_scales))


@pytest.mark.parametrize("qn,dtype,D", [(1, "bf16", 128), (4, "f16", 64), (9, "bf16", 64), (40, "f16", 128), (100, "bf16", 128),
                                        (100, "f16", 64)])
def test_device_descales_give_what_floats_give(cuda_lib, qn, dtype, D):
    """Written, read and attended to with the descales in tensors, in one of each, and as floats: bit for bit."""
    st = Step([qn, 1], [300, 257], 8, 2, D, 16, dtype, seed=qn, kd=0.0031, vd=0.0017)
    want = bits(st.run())
    slots = torch.arange(64, device="cuda")
    rows = torch.randn(64, 2, D, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    fa.kv4_write(rows, rows, slots, spare := junk_cache(4, 16, 2, D, 0.0031, 0.0017))
    codes, read = cache_bits(spare), bits(fa.kv4_read(spare, slots, DT[dtype]))
    for kd, vd in ((one(0.0031), one(0.0017)), (one(0.0031).view(()), 0.0017), (0.0031, one(0.0017))):
        st.cache.k_descale, st.cache.v_descale = kd, vd
        assert all(torch.equal(a, b) for a, b in zip(want, bits(st.run())))
        c = junk_cache(4, 16, 2, D, kd, vd)
        fa.kv4_write(rows, rows, slots, c)
        assert all(torch.equal(a, b) for a, b in zip(codes, cache_bits(c)))
        assert all(torch.equal(a, b) for a, b in zip(read, bits(fa.kv4_read(c, slots, DT[dtype]))))


@pytest.mark.parametrize("qn", [1, 9, 100])
def test_captured_calls_follow_the_device_descales(cuda_lib, qn):
    st = Step([qn], [700], 8, 2, 128, 32, "bf16", seed=qn)
    kd, vd = one(0.003), one(0.002)
    st.cache.k_descale, st.cache.v_descale = kd, vd
    rows = torch.randn(32, 2, 128, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    slots = torch.arange(32, device="cuda")
    spare = junk_cache(1, 32, 2, 128, kd, vd)
    ws = fa.paged_attention_kv4_workspace(st.q, st.cache, max_seqlen_q=qn, n_seqs=1, total_k=700)

    def calls(cache, other):
        fa.kv4_write(rows, rows, slots, other)
        return (*fa.kv4_read(other, slots), *fa.paged_attention_kv4(st.q, cache, st.cu, st.used, st.table, max_seqlen_q=qn,
                                                                    total_k=700, workspace=ws))

    calls(st.cache, spare)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(st.cache, spare)
    for a, b in ((0.003, 0.002), (0.0007, 0.01), (0.02, 0.0001)):
        kd.fill_(a)
        vd.fill_(b)
        graph.replay()
        c = st.cache
        fixed = fa.KV4Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, a, b)
        want = calls(fixed, junk_cache(1, 32, 2, 128, a, b))
        assert all(torch.equal(x, y) for x, y in zip(bits(got), bits(want)))


def test_device_descales_outside_the_range(cuda_lib):
    """They count as the range's nearer end."""
    rows = torch.randn(16, 1, 64, generator=torch.Generator().manual_seed(5)).half().cuda()
    slots = torch.arange(16, device="cuda")
    for bad, end in ((0.0, 2.0 ** -100), (-1.0, 2.0 ** -100), (float("nan"), 2.0 ** -100), (float("inf"), 2.0 ** 100), (1e-40, 2.0 ** -100)):
        a, b = junk_cache(1, 16, 1, 64, one(bad), one(bad)), junk_cache(1, 16, 1, 64, end, end)
        fa.kv4_write(rows, rows, slots, a)
        fa.kv4_write(rows, rows, slots, b)
        assert all(torch.equal(x, y) for x, y in zip(cache_bits(a), cache_bits(b)))


def test_descales_of_the_wrong_kind_are_refused(cuda_lib):
    for bad in (one(1.0).double(), one(1.0).cpu(), one(1.0).expand(2).contiguous()):
        with pytest.raises((TypeError, ValueError)):
            fa.KV4Cache.allocate(1, 16, 1, 64, k_descale=bad)
        c = fa.KV4Cache.allocate(1, 16, 1, 64)
        with pytest.raises((TypeError, ValueError)):
            c.v_descale = bad


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_read_rounds_once(cuda_lib, dtype):
    """Every code and scale under descales that put products next to (not on) ties of the type,
    where a rounding to fp32 in between takes them for the tie."""
    dt, keep = DT[dtype], {"bf16": 16, "f16": 13}[dtype]
    v = np.unique(np.outer(ref.E2M1, ref.e4m3_values()[:127]))
    v = v[(v > 0.25) & (v < 64)]
    g = np.random.default_rng(7).uniform(0.5, 1, 100000).astype(np.float32)
    p = v.astype(np.float32)[None, :] * g[:, None]
    near = ((p.view(np.uint32) & ((1 << keep) - 1)) == 1 << (keep - 1)) & (p.astype(np.float64) != v[None, :] * g[:, None].astype(np.float64))
    chosen = g[near.any(1)][:12]
    assert len(chosen) == 12
    cache = fa.KV4Cache.allocate(16, 16, 1, 64)
    # row r of page p: scale 8 p + r / 2 (no NaN), every code of both signs
    codes = torch.arange(16, dtype=torch.uint8).repeat(4).view(32, 2)
    cache.k_codes.copy_((codes[:, 0] | codes[:, 1] << 4).expand(16, 1, 16, 32))
    cache.k_scales.view(torch.uint8).copy_((torch.arange(256) // 2).clamp(max=126).to(torch.uint8).view(16, 1, 16, 1).expand(16, 1, 16, 4))
    cache.v_codes.copy_(cache.k_codes)
    cache.v_scales.copy_(cache.k_scales)
    slots = torch.arange(256, device="cuda")
    for a in chosen:
        cache.k_descale, cache.v_descale = float(a), float(a)
        k, v = fa.kv4_read(cache, slots, dtype=dt)
        assert torch.equal(k, v)
        exact = ref.values(raw(cache.k_codes), raw(cache.k_scales), a).transpose(0, 2, 1, 3).reshape(256, 1, 64)
        got = np64(k)
        # no neighbour of the result is nearer (products of 30 bits, exact in 64)
        for step in (torch.tensor(float("inf")), torch.tensor(float("-inf"))):
            other = np64(torch.nextafter(k, step.to(dt).cuda().expand_as(k)))
            assert (np.abs(got - exact) <= np.abs(other - exact)).all()


@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("qn", [1, 12, 40, 100])
def test_the_least_descale_under_large_queries(cuda_lib, qn, on_device):
    """K's descale 2^-100, made up for by bf16 queries of 1e27: ordinary scores, whichever way they go."""
    kd = 2.0 ** -100
    st = Step([qn, 1], [700, 90], 4, 2, 128, 16, "bf16", seed=31, std=1e-27, kd=kd)
    if on_device:
        st.cache.k_descale = one(kd)
    st.q.mul_(1e27)
    o, lse = st.run()
    st.cache.k_descale = kd
    st.check(o, lse)


@pytest.mark.parametrize("n", [12127, 12128, 12200, 12287, 12288, 16384])
def test_unpacking_around_48_kb_of_sums(cuda_lib, n):
    """In a process of its own: no larger launch before it has asked for shared memory.  All sequences
    share a page; each has a few of its keys, and every 50th a query."""
    code = f"""
import numpy as np, torch, tiled_attention_10_gb300 as fa
from tests import paged_reference as ref
n, g = {n}, torch.Generator().manual_seed(1)
cache = fa.KV4Cache.allocate(1, 16, 1, 64, k_descale=0.003, v_descale=0.002)
rows = [torch.randn(16, 1, 64, generator=g).half().cuda() for _ in range(2)]
slots = torch.arange(16, device="cuda")
fa.kv4_write(*rows, slots, cache)
raw = lambda t: t.view(torch.uint8).cpu().numpy()[0, 0]
k = ref.values(raw(cache.k_codes), raw(cache.k_scales), 0.003)
v = ref.values(raw(cache.v_codes), raw(cache.v_scales), 0.002)
has = torch.arange(n) % 50 == 0
cu = torch.cat((torch.zeros(1, dtype=torch.int32), has.int().cumsum(0).int())).cuda()
used = (torch.arange(n, dtype=torch.int32) % 16 + 1).cuda()
q = torch.randn(int(has.sum()), 1024, 64, generator=g).half().cuda()          # 1024 heads on one: unpacked
o, lse = fa.paged_attention_kv4(q, cache, cu, used, torch.zeros(n, 1, dtype=torch.int32, device="cuda"), max_seqlen_q=1,
                                total_k=n * 17)
lens = used.cpu()[has].numpy()
q64 = q.double().cpu().numpy()
s, reach = q64 @ k.T / 8, np.abs(q64) @ np.abs(k).T / 8                  # [rows, heads, keys]
seen = np.arange(16)[None, None, :] < lens[:, None, None]
s = np.where(seen, s, -np.inf)
top = s.max(-1, keepdims=True)
p = np.exp(s - top)
l = p.sum(-1, keepdims=True)
O, PV, L = p / l @ v, p / l @ np.abs(v), (top + np.log(l))[..., 0].T
A = np.where(seen, reach, 0).max(-1).T
bo, bl = ref.attend_bounds(O, PV, A, 16, 64, torch.float16, 2.0 ** -11, 0.0)
assert (np.abs(o.double().cpu().numpy() - O) <= bo).all()
assert (np.abs(lse.double().cpu().numpy() - L) <= bl).all()
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_whose_waits_run_out(cuda_lib, D):
    """Waits limited to less than the work takes: the kernel gives up, ends and says so, and the next
    calls are right.  (Every wait has its limit, so that nothing hangs.)"""
    steps = [Step([9] * 3, [9000, 300, 5000], 8, 2, D, 64, "bf16", seed=33), Step([32] * 40, [700] * 40, 8, 2, D, 64, "bf16", seed=34)]
    want = [st.run() for st in steps]
    assert binding.fa_last_device_error() == 0
    seen = set()
    try:
        for limit in (1, 100, 1000, 3000, 10000, 30000):
            binding.fa_set_wait_limit_ns(limit)
            for st, w in zip(steps, want):
                got = st.run()
                status = binding.fa_last_device_error()
                seen.add(status)
                assert status in ((5,) if limit == 1 else (0, 5))
                if status == 0:
                    assert torch.equal(got[0].view(torch.int16), w[0].view(torch.int16)) and torch.equal(got[1], w[1])
    finally:
        binding.fa_set_wait_limit_ns(0)
    assert 5 in seen
    for st, w in zip(steps, want):
        for _ in range(3):
            got = st.run()
            assert torch.equal(got[0].view(torch.int16), w[0].view(torch.int16)) and torch.equal(got[1], w[1])
    assert binding.fa_last_device_error() == 0


# ---------------------------------------------------------------- the way's own rounding of P
def is_unpacked(st, max_q):
    """Whether a call goes through unpacked rows (P in the queries' type) by the library's rule;
    otherwise P is held in f16."""
    rows = max_q * (st.H // st.H_kv)
    return rows > (512 if sum(st.seq_k) // 2048 >= len(st.seq_k) else 128)


@pytest.mark.parametrize("scale", [-0.08, 0.0, 1.0, 3.0])
@pytest.mark.parametrize("qn,keys", [(40, (900, 333)), (64, (900, 333)), (65, (900, 333)), (200, (4000, 3000))])
def test_scales_by_the_ways_bound(cuda_lib, scale, qn, keys):
    st = Step([qn, qn - 3], list(keys), 4, 2, 128, 16, "bf16", seed=41)
    st.check(*st.run(scale=scale), scale=scale, unpacked=is_unpacked(st, qn))


@pytest.mark.parametrize("qn", [12, 40, 64, 65, 100])
def test_bad_pages_by_the_ways_bound(cuda_lib, qn):
    st = Step([qn, qn], [100, 70], 4, 2, 128, 16, "bf16", seed=42, bad_page=True)
    st.check(*st.run(), unpacked=is_unpacked(st, qn))


@pytest.mark.parametrize("std,mul", [(30.0, 1.0), (1.0, 1e-30), (1.0, 1e30), (1e-3, 1.0)])
@pytest.mark.parametrize("qn", [20, 32, 33])
def test_magnitudes_by_the_ways_bound(cuda_lib, std, mul, qn):
    st = Step([qn, 12, 2], [700, 64, 90], 4, 1, 128, 32, "bf16", seed=43, std=std, kd=0.003 * std)
    st.q.mul_(mul)
    scale = 128 ** -0.5 / mul
    st.check(*st.run(scale=scale), scale=scale, unpacked=is_unpacked(st, qn))


# One page, every table entry that page, and as many keys as a call takes: attention over it is
# attention over the page alone, lse apart by log of the number of times.
@pytest.mark.parametrize("qn,ps,rest", [(1, 128, 0), (1, 128, 31), (2, 128, 0), (2, 128, 100), (5, 128, 0), (5, 6016, 0), (1, 6016, 0)])
def test_sequences_up_to_two_billion_keys(cuda_lib, qn, ps, rest):
    most = (1 << 31) - 256
    cols = most // ps
    assert cols * ps == most                        # both page sizes divide it
    g = torch.Generator().manual_seed(qn + ps)
    cache = fa.KV4Cache.allocate(1, ps, 1, 64, k_descale=0.003, v_descale=0.002)
    rows = [torch.randn(ps, 1, 64, generator=g).bfloat16().cuda() for _ in range(2)]
    fa.kv4_write(*rows, torch.arange(ps, device="cuda"), cache)
    q = torch.randn(qn, 8, 64, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, qn], dtype=torch.int32, device="cuda")
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    n = most - rest
    o, lse = fa.paged_attention_kv4(q, cache, cu, torch.tensor([n], dtype=torch.int32, device="cuda"), table, max_seqlen_q=qn,
                                    causal="none")
    assert binding.fa_last_device_error() == 0
    k, v = (ref.gather(raw(a), raw(b), d, [0], ps, 1) for a, b, d in ((cache.k_codes, cache.k_scales, 0.003),
                                                                      (cache.v_codes, cache.v_scales, 0.002)))
    O, L, PV, A = ref.attend(np64(q), k, v, 64 ** -0.5, 0)
    # The cut page changes O by no more than its share of the keys.  Sums over so many keys lose 2^-24
    # an add, the matrix unit's perhaps twice that (its rounding is not documented): up to 16 rows 1824
    # warps take 32 keys a step, 4 adds to a lane's sum and 2 products; above, 152 blocks take 128 keys,
    # one add and 8 products.
    steps = n / 32 / 1824 if qn * 8 <= 16 else n / 128 / 152
    sums, products = (4 * steps, 2 * steps) if qn * 8 <= 16 else (steps, 8 * steps)
    bo, bl = ref.attend_bounds(O, PV, A, ps, 64, torch.bfloat16, ref.half_step(torch.float16), 0.0)
    loss, share = sums * 2.0 ** -24, 2.0 * ps / n
    assert (np.abs(np64(o) - O) <= bo + (loss + products * 2.0 ** -23 + share) * (PV + np.abs(O))).all()
    assert (np.abs(np64(lse) - (L + np.log(n / ps))) <= bl + loss + share + 2.0 ** -24 * 22).all()


def test_no_descales_are_ones(cuda_lib):
    """Null device descales: 1."""
    a, b = junk_cache(2, 16, 1, 64, 1.0, 1.0), junk_cache(2, 16, 1, 64, 1.0, 1.0)
    x = torch.randn(20, 1, 64, generator=torch.Generator().manual_seed(6)).half().cuda() * 100
    slots, stream = torch.arange(20, device="cuda"), torch.cuda.current_stream().cuda_stream
    fa.kv4_write(x, x, slots, a)
    ptrs = [t.data_ptr() for t in (b.k_codes, b.k_scales, b.v_codes, b.v_scales)]
    assert binding.fa_kv4_write_devscale(x.data_ptr(), x.data_ptr(), slots.data_ptr(), *ptrs, None, None, 20, 1, 64, 16, 2,
                                         [(64, 64, 64)] * 2, "f16", stream) == 0
    assert all(torch.equal(s, t) for s, t in zip(cache_bits(a), cache_bits(b)))
    k, v = torch.empty_like(x), torch.empty_like(x)
    assert binding.fa_kv4_read_devscale(*ptrs, slots.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, 20, 1, 64, 16, 2, "f16",
                                        stream) == 0
    assert all(torch.equal(s, t) for s, t in zip(fa.kv4_read(a, slots, torch.float16), (k, v)))


def test_queries_past_32_bit_offsets(cuda_lib):
    """300,000 requests of one token each: rows of q and O, and of the table, far beyond 2^32 bytes."""
    n, H, D = 300_000, 64, 128
    g = torch.Generator().manual_seed(51)
    cache = fa.KV4Cache.allocate(3, 16, 8, D, k_descale=0.003, v_descale=0.002)
    rows = [torch.randn(48, 8, D, generator=g).bfloat16().cuda() for _ in range(2)]
    fa.kv4_write(*rows, torch.arange(48, device="cuda"), cache)
    q = torch.randn(n, H, D, generator=torch.Generator(device="cuda").manual_seed(52), device="cuda", dtype=torch.bfloat16)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    used = torch.arange(n, dtype=torch.int32, device="cuda") % 33
    table = (torch.arange(2 * n, dtype=torch.int32, device="cuda") % 3).view(n, 2).contiguous()
    used.clamp_(max=32)
    o, lse = fa.paged_attention_kv4(q, cache, cu, used, table, max_seqlen_q=1, total_k=32 * n)
    for a in (0, 140_000, n - 70):
        part = slice(a, a + 70)
        o2, l2 = fa.paged_attention_kv4(q[part].contiguous(), cache, cu[:71].contiguous(), used[part].contiguous(), table[part].contiguous(),
                                        max_seqlen_q=1, total_k=32 * 70)
        # one chunk of keys each: no request is cut, whatever the split of the work
        assert torch.equal(o[part], o2) and torch.equal(lse[:, part], l2)


def test_write_rows_far_apart(cuda_lib):
    """Token and head strides that pass 2^32 elements."""
    g = torch.Generator().manual_seed(53)
    near = [torch.randn(3, 2, 64, generator=g).half().cuda() for _ in range(2)]
    step = (1 << 32) + 64
    buf = torch.empty(2 * step + 4096, dtype=torch.float16, device="cuda")
    far = buf.as_strided((3, 2, 64), (step, 1024, 1))
    wide = buf.as_strided((3, 2, 64), (512, step, 1), 2048)
    slots = torch.arange(3, device="cuda")
    for view in (far, wide):
        a, b = junk_cache(1, 16, 2, 64, 0.003, 0.002), junk_cache(1, 16, 2, 64, 0.003, 0.002)
        view.copy_(near[0])
        fa.kv4_write(view, view, slots, a)
        fa.kv4_write(near[0], near[0], slots, b)
        assert all(torch.equal(x, y) for x, y in zip(cache_bits(a), cache_bits(b)))
