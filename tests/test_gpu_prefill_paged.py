"""Ragged prefill over page pools (fa_prefill_paged) against the f64 oracle, every element.  Slots
that hold no token are NaN throughout, so a result that touched one would show it.  Tolerance:
gpu_common.check_close -- the kernel rounds P once before the PV contraction, a q4_0 side once when
dequantized and O once when stored, as the prefill kernels it is stated for."""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import UNIT_ROUNDOFF, check_close, np64
from paged_common import DT, make_ragged, q4_buffer, q4_planes

pytestmark = pytest.mark.gpu


def make_q(rows, Hq, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, Hq, D, generator=g).to(DT[dtype])


def expected(r, q, causal=True, scale=None):
    """{sequence: [n, Hq, D] f64}; rows that see no key are zeros."""
    out = {}
    D = q.shape[-1]
    for b, (n, length) in enumerate(zip(r.new, r.lens)):
        if n == 0:
            continue
        s = int(r.starts[b])
        want = np.zeros((n, q.shape[1], D))
        blind = min(n, max(0, n - length) if causal else (n if length == 0 else 0))
        if blind < n:
            qs = np64(q[s + blind:s + n]).transpose(1, 0, 2)[None]
            o = oracle.attention(np.ascontiguousarray(qs), r.sequence("k", b)[None],
                                 r.sequence("v", b)[None], causal=causal,
                                 q_pos_offset=max(0, length - n) if causal else 0,
                                 scale=scale or D ** -0.5)
            want[blind:] = o[0].transpose(1, 0, 2)
        out[b] = want
    return out


def check(r, q, o, causal=True, scale=None):
    q4 = "q4_0" in (r.kf, r.vf)
    for b, want in expected(r, q, causal, scale).items():
        s = int(r.starts[b])
        got = np64(o[s:s + r.new[b]])
        blind = np.all(want == 0, axis=-1)
        assert (got[blind] == 0).all(), f"sequence {b}: a row without keys is not zero"
        check_close(got[~blind], want[~blind], r.dtype, f"sequence {b} ({r.new[b]} of {r.lens[b]})",
                    q4=q4)


def run(fa, r, q, **kw):
    o = fa.fa_prefill_paged(q.cuda(), r.pool(fa, "k"), r.pool(fa, "v"), *r.batch(), **kw)
    assert fa.fa_get_status() == fa.FA_OK
    return o


CASES = [
    # new, lens, Hq, Hkv, D, page, dtype, kf, vf
    ([1], [1], 8, 2, 128, 128, "f16", "dense", "dense"),
    ([1], [1], 8, 2, 128, 128, "f16", "q4_0", "q4_0"),
    ([5], [133], 8, 2, 128, 64, "f16", "dense", "dense"),
    ([40], [300], 8, 2, 128, 128, "bf16", "q4_0", "q4_0"),
    ([200], [200], 8, 8, 64, 16, "bf16", "dense", "dense"),
    ([1, 0, 300, 1, 17], [777, 50, 300, 1, 1029], 32, 8, 128, 16, "f16", "dense", "dense"),
    ([1, 0, 300, 1, 17], [777, 50, 300, 1, 1029], 32, 8, 128, 128, "f16", "q4_0", "q4_0"),
    ([64, 65, 63, 1, 128, 129], [64, 1000, 63, 4096, 256, 1300], 16, 2, 64, 128, "f16", "q4_0",
     "dense"),
    ([33, 1, 500], [1111, 2, 700], 12, 4, 128, 48, "bf16", "dense", "q4_0"),
    ([7, 90], [5000, 91], 20, 4, 128, 32, "f16", "q4_0", "dense"),
    ([257, 3], [600, 3], 7, 1, 64, 256, "bf16", "q4_0", "q4_0"),
    ([31, 2], [2049, 129], 48, 1, 128, 64, "f16", "dense", "dense"),
    ([3, 2], [513, 40], 128, 1, 64, 16, "f16", "dense", "q4_0"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[2:])) + f"-{c[0]}")
def test_matches_oracle(fa, case):
    new, lens, Hq, Hkv, D, page, dtype, kf, vf = case
    r = make_ragged(new, lens, Hkv, D, page, dtype, kf, vf, seed=sum(lens) + page)
    q = make_q(sum(new), Hq, D, dtype, seed=3)
    check(r, q, run(fa, r, q))


@pytest.mark.parametrize("kf,vf", [("dense", "dense"), ("q4_0", "q4_0")])
def test_many_short_sequences(fa, kf, vf):
    """More units than CTAs times any queue: 150 sequences of a few keys, so that a CTA's run holds
    many segments."""
    rng = np.random.default_rng(7)
    new = [int(x) for x in rng.integers(0, 4, 150)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 200, 150))]
    r = make_ragged(new, lens, 8, 128, 128, "f16", kf, vf, seed=11)
    q = make_q(sum(new), 32, 128, "f16", seed=12)
    check(r, q, run(fa, r, q))


@pytest.mark.parametrize("kf,vf", [("dense", "dense"), ("q4_0", "dense"), ("q4_0", "q4_0")])
def test_one_long_sequence_split_over_all_ctas(fa, kf, vf):
    """One token over 40 000 keys and one kv head: the unit is cut into a piece per CTA."""
    r = make_ragged([1], [40003], 1, 128, 128, "bf16", kf, vf, seed=21)
    q = make_q(1, 4, 128, "bf16", seed=22)
    check(r, q, run(fa, r, q))


@pytest.mark.parametrize("kf", ["dense", "q4_0"])
def test_rows_without_keys_are_zero(fa, kf):
    """More rows than tokens (positions below 0) and sequences without any key."""
    r = make_ragged([5, 3, 200, 2], [2, 0, 60, 900], 2, 64, 128, "f16", kf, kf, seed=31)
    q = make_q(210, 8, 64, "f16", seed=32)
    check(r, q, run(fa, r, q))
    r0 = make_ragged([4, 1], [0, 0], 2, 64, 128, "f16", kf, kf, seed=33)
    o = run(fa, r0, make_q(5, 8, 64, "f16", seed=34), o=torch.ones(5, 8, 64).half().cuda())
    assert (o == 0).all()


@pytest.mark.parametrize("kf,vf", [("dense", "dense"), ("q4_0", "q4_0")])
def test_without_the_causal_mask(fa, kf, vf):
    r = make_ragged([70, 1, 3, 2], [300, 129, 1, 0], 2, 128, 64 if kf == "dense" else 128, "f16",
                    kf, vf, seed=41)
    q = make_q(76, 8, 128, "f16", seed=42)
    check(r, q, run(fa, r, q, causal=False, scale=0.03), causal=False, scale=0.03)


def test_score_ramp_moves_frames(fa):
    """Scores that grow by 2 a key block push the rows' frames past the 10-point margin every few
    blocks, also across the pieces of units cut between CTAs."""
    n, length, D = 300, 6000, 128
    r = make_ragged([n], [length], 2, D, 128, "f16", "dense", "dense", seed=51, poison=False)
    for p in range(r.table.shape[1]):
        r.k[int(r.table[0, p]), :, :, 0] = 2.0 * p / (8.0 * D ** -0.5)
    q = make_q(n, 8, D, "f16", seed=52)
    q[..., 0] = 8.0
    check(r, q, run(fa, r, q))


def test_strides_and_padding(fa):
    """q cut out of a fused projection, o head-major, rows before the first sequence and behind the
    last one: those rows stay as they were."""
    new, lens, Hq, Hkv, D = [9, 1, 30], [200, 77, 30], 8, 2, 128
    first, pad = 3, 6
    rows = first + sum(new) + pad
    r = make_ragged(new, lens, Hkv, D, 64, "f16", "dense", "dense", seed=61, first_row=first)
    fused = make_q(rows, Hq + 2 * Hkv, D, "f16", seed=62).cuda()
    q = fused[:, :Hq]
    o = torch.full((Hq, rows, D), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    out = fa.fa_prefill_paged(q, r.pool(fa, "k"), r.pool(fa, "v"), *r.batch(), o)
    assert fa.fa_get_status() == fa.FA_OK and out is o
    check(r, q.cpu(), o.cpu())
    assert (o[:first] == 7.0).all() and (o[first + sum(new):] == 7.0).all()
    dense = fa.fa_prefill_paged(q.contiguous(), r.pool(fa, "k"), r.pool(fa, "v"), *r.batch())
    assert torch.equal(dense[first:first + sum(new)], o[first:first + sum(new)])
    assert (dense[:first] == 0).all() and (dense[first + sum(new):] == 0).all()


def test_agrees_with_the_contiguous_prefill_and_the_paged_decode(fa):
    """One chunk over pages in order is fa_fwd's chunk over the same cache; one token per sequence is
    fa_decode_paged's call.  Both kernels are compared with the same oracle elsewhere; here within
    twice its bound, u = 2^-11 on each side."""
    D, page = 128, 128
    r = make_ragged([260], [1500], 2, D, page, "f16", "dense", "dense", seed=71, poison=False)
    q = make_q(260, 8, D, "f16", seed=72).cuda()
    o = run(fa, r, q)
    k, v = (torch.from_numpy(r.sequence(s, 0)).half().cuda()[None].contiguous() for s in "kv")
    ref = fa.fa_fwd(q.transpose(0, 1)[None].contiguous(), k, v)[0].transpose(0, 1)
    want = expected(r, q.cpu())[0]
    rms = np.sqrt(np.mean(want ** 2, -1, keepdims=True))
    assert (np.abs(np64(o) - np64(ref)) <= 2 * 2.0 ** -11 * (np.abs(want) + 6 * rms)).all()
    r = make_ragged([1] * 5, [300, 1, 129, 2000, 128], 2, D, page, "f16", "q4_0", "q4_0", seed=73)
    q = make_q(5, 8, D, "f16", seed=74).cuda()
    o = run(fa, r, q)
    table, _, lens = r.batch()
    ref = fa.fa_decode_paged(q[:, :, None].contiguous(), r.pool(fa, "k"), r.pool(fa, "v"), table,
                             lens)[:, :, 0]
    for b, want in expected(r, q.cpu()).items():
        rms = np.sqrt(np.mean(want ** 2, -1, keepdims=True))
        assert (np.abs(np64(o[b:b + 1]) - np64(ref[b:b + 1]))
                <= 2 * 2.0 ** -11 * (np.abs(want) + 9 * rms)).all()


def test_repeated_calls_are_bitwise_equal_with_a_stale_workspace(fa):
    r = make_ragged([1, 300, 1, 40], [5000, 4000, 3, 900], 8, 128, 128, "f16", "dense", "dense",
                    seed=81)
    q = make_q(342, 32, 128, "f16", seed=82).cuda()
    k, v, batch = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
    ws = torch.full((fa.fa_prefill_paged_workspace_bytes(32, 8, 128),), 255, dtype=torch.uint8,
                    device="cuda")
    first = fa.fa_prefill_paged(q, k, v, *batch, workspace=ws)
    check(r, q.cpu(), first.cpu())
    for _ in range(8):
        assert torch.equal(first, fa.fa_prefill_paged(q, k, v, *batch, workspace=ws))
    assert fa.fa_get_status() == fa.FA_OK


@pytest.mark.parametrize("D,kf,vf,heads", [
    (64, "dense", "q4_0", (8, 8)), (64, "q4_0", "q4_0", (8, 2)), (64, "q4_0", "dense", (14, 2)),
    (64, "dense", "dense", (3, 3)), (128, "q4_0", "dense", (8, 8)), (128, "q4_0", "q4_0", (28, 4)),
    (128, "dense", "q4_0", (8, 2)), (128, "dense", "dense", (10, 2))])
def test_units_cut_between_ctas(fa, D, kf, vf, heads):
    """Prompts, chunks and single tokens whose units are cut into two to many pieces, merged by
    whichever CTA comes last: every launch gives the same bytes."""
    Hq, Hkv = heads
    r = make_ragged([333, 1, 1021, 77, 600, 2], [333, 1500, 1400, 2100, 6000, 1030], Hkv, D, 64,
                    "f16", kf, vf, seed=85)
    q = make_q(sum(r.new), Hq, D, "f16", seed=86).cuda()
    k, v, batch = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
    first = fa.fa_prefill_paged(q, k, v, *batch)
    check(r, q.cpu(), first.cpu())
    o = torch.empty_like(first)
    for _ in range(60):
        o.fill_(7.0)
        assert torch.equal(first, fa.fa_prefill_paged(q, k, v, *batch, o))
    assert fa.fa_get_status() == fa.FA_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (3, 1), (4, 2), (5, 1), (8, 1), (16, 1), (64, 1)])
def test_one_token_over_many_pieces(fa, D, heads):
    """Pieces of a few rows: the merge's threads share a row."""
    Hq, Hkv = heads
    for new, length, seed in (([1], [9000], 87), ([2], [3001], 88)):
        r = make_ragged(new, length, Hkv, D, 64, "bf16", "dense", "q4_0", seed=seed)
        q = make_q(new[0], Hq, D, "bf16", seed=seed + 10)
        check(r, q, run(fa, r, q.cuda()).cpu())


def test_more_sequences_than_a_warp(fa):
    """The run is located 32 sequences at a time; empty ones among them."""
    new = [(7 * i) % 5 for i in range(75)]
    lens = [n + (311 * i) % 1700 for i, n in enumerate(new)]
    r = make_ragged(new, lens, 2, 64, 64, "f16", "dense", "dense", seed=89)
    q = make_q(sum(new), 8, 64, "f16", seed=90)
    check(r, q, run(fa, r, q.cuda()).cpu())


def test_captured_call_serves_other_batches(fa):
    """A captured call replayed after row_starts, seq_lens, the table and q were rewritten, and a
    second graph over the same workspace in between."""
    D = 128
    batches = [([1, 200, 0, 7], [900, 200, 5, 2000]), ([3, 3, 201, 1], [3, 4000, 300, 1]),
               ([0, 0, 1, 0], [0, 0, 640, 0])]
    rs = [make_ragged(n, l_, 8, D, 128, "bf16", "q4_0", "dense", seed=90 + i, spare=60 - sum(
        -(-x // 128) for x in l_)) for i, (n, l_) in enumerate(batches)]
    pps = max(r.table.shape[1] for r in rs)
    rows = 208
    q = torch.zeros(rows, 32, D, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    o2 = torch.zeros_like(q)
    k, v = rs[0].pool(fa, "k"), rs[0].pool(fa, "v")
    table = torch.zeros(4, pps, dtype=torch.int32, device="cuda")
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fa_prefill_paged_workspace_bytes(32, 8, D), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    graphs = []
    for out in (o, o2):
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            fa.fa_prefill_paged(q, k, v, table, starts, lens, out, workspace=ws)
        graphs.append(g)
    for i, r in enumerate(rs + rs[:1]):
        x = make_q(rows, 32, D, "bf16", seed=95 + i)
        q.copy_(x)
        k.buf.copy_(r.k)
        v.copy_(r.v)
        table.zero_()
        table[:, :r.table.shape[1]] = r.table.cuda()
        starts.copy_(r.starts)
        lens.copy_(torch.tensor(r.lens, dtype=torch.int32))
        o.fill_(5.0)
        o2.fill_(5.0)
        for g in graphs:
            g.replay()
        assert fa.fa_get_status() == fa.FA_OK
        check(r, x, o.cpu())
        assert torch.equal(o, o2) and (o[sum(r.new):] == 5.0).all()


def test_other_stream_allocates_there(fa):
    r = make_ragged([300], [4000], 8, 128, 128, "f16", "dense", "dense", seed=101)
    q, k, v, batch = (make_q(300, 32, 128, "f16", seed=102).cuda(), r.pool(fa, "k"),
                      r.pool(fa, "v"), r.batch())
    want = fa.fa_prefill_paged(q, k, v, *batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append(fa.fa_prefill_paged(q, k, v, *batch, stream=side))
        torch.empty(50 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # the other stream's
    outs.append(fa.fa_prefill_paged(q, k, v, *batch, stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def test_bad_batches_are_reported(fa):
    """Row starts out of order or past the tensors: nothing is written.  A page outside the pool and a
    length past the table: recorded, the rest of the batch is right."""
    r = make_ragged([4, 9], [300, 200], 2, 128, 128, "f16", "dense", "dense", seed=111)
    q = make_q(13, 8, 128, "f16", seed=112).cuda()
    k, v, (table, starts, lens) = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
    for bad in ([0, 9, 4], [-1, 4, 13], [0, 4, 14], [5, 4, 13]):
        o = torch.full_like(q, 3.0)
        fa.fa_prefill_paged(q, k, v, table, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                            lens, o)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        assert (o == 3.0).all()
    for page in (r.shape[0], -1, 1 << 30):
        t = table.clone()
        t[0, 1] = page
        o = fa.fa_prefill_paged(q, k, v, t, starts, lens)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        check_close(np64(o[4:]), expected(r, q.cpu())[1], "f16", "the other sequence")
    for n in (-1, 128 * table.shape[1] + 1):
        o = fa.fa_prefill_paged(q, k, v, table, starts,
                                torch.tensor([n, 200], dtype=torch.int32, device="cuda"))
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        check_close(np64(o[4:]), expected(r, q.cpu())[1], "f16", "the other sequence")
    o = fa.fa_prefill_paged(q, k, v, table, starts, lens)
    assert fa.fa_get_status() == fa.FA_OK


def test_no_rows(fa):
    r = make_ragged([0, 0], [5, 0], 2, 128, 128, "f16", "dense", "dense", seed=121)
    o = run(fa, r, make_q(0, 8, 128, "f16", seed=122))
    assert o.shape == (0, 8, 128)
    o = run(fa, r, make_q(3, 8, 128, "f16", seed=123))  # padding only
    assert (o == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_is_dequantized_as_read(fa, dtype, D):
    """One key a sequence has weight 1 whatever its (here zero) score: o is the value row itself, for
    every finite scale and all codes what fa_read_paged gives, products past the type's range
    included."""
    Hkv, page = 8, 16
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    scales = every[torch.isfinite(every.view(torch.float16))]
    blocks = Hkv * D // 32
    B = -(-scales.numel() // blocks)
    g = torch.Generator().manual_seed(131)
    buf = torch.zeros(fa.fa_q4_0_bytes(B, Hkv, page, D), dtype=torch.uint8)
    nib, sc = q4_planes(buf, (B, Hkv, page, D))
    nib.copy_(torch.randint(256, nib.shape, generator=g, dtype=torch.uint8))
    sc[:, :, 0] = scales.repeat(2)[:B * blocks].view(B, Hkv, D // 32)
    pool = fa.Q4Tensor(buf.cuda(), B, Hkv, page, D)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    q = make_q(B, Hkv, D, dtype, seed=132).cuda()
    zeros = torch.zeros(B, Hkv, page, D, dtype=DT[dtype])
    keys = fa.Q4Tensor(q4_buffer(zeros).cuda(), B, Hkv, page, D)
    want = torch.empty_like(q)
    fa.fa_read_paged(pool, None, table, starts, lens, want)
    assert fa.fa_get_status() == fa.FA_OK
    for k in (keys, zeros.cuda()):
        assert torch.equal(fa.fa_prefill_paged(q, k, pool, table, starts, lens), want)
    assert fa.fa_get_status() == fa.FA_OK


@pytest.mark.parametrize("kf,vf", [("dense", "dense"), ("q4_0", "q4_0"), ("dense", "q4_0")])
def test_rows_of_no_sequence_may_hold_anything(fa, kf, vf):
    """NaN and infinities in q's rows before, behind and (an unused head's place) beside the batch:
    tiles load some of them along with a sequence's rows."""
    new, lens = [70, 1, 33], [900, 1500, 33]
    r = make_ragged(new, lens, 2, 128, 64, "f16", kf, vf, seed=141, first_row=5)
    rows = 5 + sum(new) + 40
    q = make_q(rows, 6, 128, "f16", seed=142)
    clean = fa.fa_prefill_paged(q.cuda(), r.pool(fa, "k"), r.pool(fa, "v"), *r.batch())
    bad = q.clone()
    bad[:5], bad[5 + sum(new):] = float("nan"), float("inf")
    wide = torch.full((rows, 8, 128), float("nan"), dtype=torch.float16)
    wide[:, 1:7] = bad
    o = fa.fa_prefill_paged(wide.cuda()[:, 1:7], r.pool(fa, "k"), r.pool(fa, "v"), *r.batch())
    assert fa.fa_get_status() == fa.FA_OK
    check(r, q, o.cpu())
    assert torch.equal(o, clean)


def test_calls_on_several_streams_at_once(fa):
    """Batches of different shapes in flight together, each with scratch of its own."""
    jobs = []
    for i, (new, lens, kf) in enumerate([([300, 1], [5000, 3000], "dense"), ([1] * 6, [2500] * 6, "q4_0"),
                                         ([90, 90], [4000, 90], "q4_0")]):
        r = make_ragged(new, lens, 8, 128, 128, "f16", kf, kf, seed=151 + i)
        args = (make_q(sum(new), 32, 128, "f16", seed=161 + i).cuda(), r.pool(fa, "k"),
                r.pool(fa, "v"), *r.batch())
        jobs.append((args, fa.fa_prefill_paged(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        outs = [fa.fa_prefill_paged(*args, stream=s) for args, _, s in jobs]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o, (_, want, _) in zip(outs, jobs))
    assert fa.fa_get_status() == fa.FA_OK


def test_append_attend_and_read_as_a_server_does(fa):
    """Prompts, then steps of one and of several tokens, written into q4_0 and dense pools and
    attended from them, pages handed out as the sequences grow; what was attended is what is read
    back."""
    Hq, Hkv, D, page, B = 8, 2, 64, 32, 3
    g = torch.Generator().manual_seed(171)
    shape = (40, Hkv, page, D)
    pools = {"k": fa.Q4Tensor(q4_buffer(torch.zeros(shape, dtype=torch.float16)).cuda(), *shape),
             "v": torch.full(shape, float("nan"), dtype=torch.float16, device="cuda")}
    free = torch.randperm(shape[0], generator=g).tolist()
    table = torch.zeros(B, 12, dtype=torch.int32)
    lens, held = [0] * B, [0] * B
    for new in ([70, 33, 1], [1, 1, 1], [1, 4, 0], [5, 1, 100], [1, 1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        for b in range(B):
            while held[b] * page < lens[b]:
                table[b, held[b]] = free.pop()
                held[b] += 1
        batch = (table.cuda(), torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32,
                                            device="cuda"),
                 torch.tensor(lens, dtype=torch.int32, device="cuda"))
        q, k_new, v_new = (torch.randn(sum(new), h, D, generator=g).half().cuda()
                           for h in (Hq, Hkv, Hkv))
        fa.fa_append_paged(k_new, v_new, pools["k"], pools["v"], *batch)
        o = fa.fa_prefill_paged(q, pools["k"], pools["v"], *batch)
        # every sequence taken out of the pages whole, then attended in 64 bits
        whole = (batch[0], torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32,
                                        device="cuda"), batch[2])
        keys, values = (torch.empty(sum(lens), Hkv, D, dtype=torch.float16, device="cuda")
                        for _ in "kv")
        fa.fa_read_paged(pools["k"], pools["v"], *whole, keys, values)
        assert fa.fa_get_status() == fa.FA_OK
        at = row = 0
        for b in range(B):
            if new[b]:
                rows = slice(row, row + new[b])
                assert torch.equal(values[at + lens[b] - new[b]:at + lens[b]], v_new[rows])
                kk, vv = (np64(x[at:at + lens[b]]).transpose(1, 0, 2)[None] for x in (keys, values))
                want = oracle.attention(np.ascontiguousarray(np64(q[rows]).transpose(1, 0, 2)[None]),
                                        np.ascontiguousarray(kk), np.ascontiguousarray(vv),
                                        causal=True, q_pos_offset=lens[b] - new[b], scale=D ** -0.5)
                check_close(np64(o[rows]), want[0].transpose(1, 0, 2), "f16", f"step {new}, {b}")
            at, row = at + lens[b], row + new[b]


@pytest.mark.parametrize("D,kf,vf", [(64, "dense", "q4_0"), (64, "q4_0", "q4_0"), (128, "q4_0", "dense"),
                                     (128, "q4_0", "q4_0"), (128, "dense", "dense")])
def test_nothing_beside_the_workspace_and_the_rows_is_written(fa, D, kf, vf):
    """Guard bytes around the scratch and around o's rows, over many launches of a batch whose units are
    cut: its prompts' units begin at token 512 among others."""
    r = make_ragged([333, 1, 1021, 77, 600], [333, 1, 1021, 77, 600], 8, D, 128, "f16", kf, vf, seed=181)
    n = sum(r.new)
    q = make_q(n, 8, D, "f16", seed=182).cuda()
    k, v, batch = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
    need, guard = fa.fa_prefill_paged_workspace_bytes(8, 8, D), 1 << 20
    scratch = torch.full((need + 2 * guard,), 90, dtype=torch.uint8, device="cuda")
    ws = scratch[guard:guard + need]
    rows = torch.full((n + 64, 8, D), 7.0, dtype=torch.float16, device="cuda")
    o = rows[32:32 + n]
    want = fa.fa_prefill_paged(q, k, v, *batch)
    check(r, q.cpu(), want.cpu())
    for _ in range(300):
        o.fill_(7.0)
        fa.fa_prefill_paged(q, k, v, *batch, o, workspace=ws)
        assert torch.equal(o, want)
    assert fa.fa_get_status() == fa.FA_OK
    assert (scratch[:guard] == 90).all() and (scratch[guard + need:] == 90).all()
    assert (rows[:32] == 7.0).all() and (rows[32 + n:] == 7.0).all()


NAN_CASES = [(kf, vf, dtype, D)
             for kf, vf in (("dense", "dense"), ("q4_0", "q4_0"), ("q4_0", "dense"))
             for dtype, D in (("f16", 128), ("bf16", 64))]


@pytest.mark.parametrize("kf,vf,dtype,D", NAN_CASES)
def test_nan_in_a_row_stays_in_that_row(fa, kf, vf, dtype, D):
    """A NaN in one query row and head makes that row's output NaN, in whole units and in units cut into two
    and more pieces; every other row keeps its bits, and rows without keys are zeros whatever they hold."""
    r = make_ragged([3, 70, 1, 40, 2, 1], [500, 70, 9000, 3000, 1, 0], 2, D, 64, dtype, kf, vf, seed=191)
    q = make_q(sum(r.new), 8, D, dtype, seed=192)
    clean = run(fa, r, q)
    check(r, q, clean.cpu())
    bad = q.clone()
    rows = {0: 1, 5: 0, 3 + 69: 7, 73: 2, 74: 3, 74 + 39: 6, 114: 4, 115: 5, 116: 1}
    for t, h in rows.items():
        bad[t, h, 5] = float("nan")
    o = run(fa, r, bad)
    for t, h in rows.items():
        seq = int((r.starts[1:] <= t).sum())
        blind = r.lens[seq] - (int(r.starts[seq + 1]) - t) < 0
        if blind:
            assert (o[t, h] == 0).all(), t
        else:
            assert torch.isnan(o[t, h]).all(), t
        o[t, h] = clean[t, h]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("kf,vf,dtype,D", NAN_CASES)
@pytest.mark.parametrize("at", [0, 768, 4096, 8960])
def test_nan_in_a_key_reaches_every_row_that_sees_it(fa, kf, vf, dtype, D, at):
    """One token over 9000 keys, a unit of many pieces: a key of NaN (a q4_0 key's scales) makes the row NaN
    whichever piece it lies in, and also where all keys of a piece are NaN."""
    for width in (1, 128, 1000):
        r = make_ragged([1], [9000], 1, D, 64, dtype, kf, vf, seed=193)
        for p in range(at, min(9000, at + width)):
            page, slot = int(r.table[0, p // 64]), p % 64
            if kf == "dense":
                r.k[page, :, slot] = float("nan")
            else:
                q4_planes(r.k, r.shape)[1][page, :, slot] = 0x7E00
        q = make_q(1, 4, D, dtype, seed=194)
        assert torch.isnan(run(fa, r, q)).all()


RAMPS = [(n, kf, vf, dtype, D)
         for n in (1, 5) for kf, vf in (("dense", "dense"), ("q4_0", "q4_0"), ("q4_0", "dense"))
         for dtype in ("f16", "bf16") for D in (64, 128)]
RAMPS += [(300, "dense", "dense", "bf16", 64), (300, "q4_0", "q4_0", "f16", 128),
          (300, "dense", "q4_0", "bf16", 128), (300, "q4_0", "q4_0", "bf16", 64)]


def check_ramp(r, q, o):
    """Every element within the sum of the roundings' worst cases, for rows whose softmax rests on a few keys
    (their outputs are as large as single values, for which check_close's absolute bar, stated for sums over
    many keys, is too small: at |o| = 4 one rounding to bf16 alone is 4 * 2^-8 = 1.6e-2).  With u half a step
    of the dtype, o = sum_j w_j v_j and A = sum_j w_j |v_j|:
      o is rounded once                                     u |o|
      P is rounded once, below 2^-14 by at most 2^-25       u A + n 2^-25 max|v|
      a q4_0 value of V is rounded once                     u A
      scores off by e move each w_j by a factor e at most
      and their sum as well                                 e (A + |o|)
    e is 2^-10 for the f32 accumulation (see the test) plus, for a q4_0 K, whose elements are rounded once,
    scale u max_j sum_{i > 0} |q_i k_ji|.  (Element 0, the ramp, is exact: it is its block's largest, its
    scale an eighth of it, and -8 times that the value again.)"""
    u, scale = UNIT_ROUNDOFF[r.dtype], q.shape[-1] ** -0.5
    for b, want in expected(r, q).items():
        s, n, length = int(r.starts[b]), r.new[b], r.lens[b]
        k, v = r.sequence("k", b), r.sequence("v", b)
        qs = np64(q[s:s + n]).transpose(1, 0, 2)
        size = oracle.attention(np.ascontiguousarray(qs[None]), k[None], np.ascontiguousarray(np.abs(v)[None]),
                                causal=True, q_pos_offset=length - n, scale=scale)[0]
        size, mag = size.transpose(1, 0, 2), np.abs(want)
        e = np.full((n, qs.shape[0], 1), 2.0 ** -10)
        if r.kf == "q4_0":
            group = qs.shape[0] // k.shape[0]
            for h in range(qs.shape[0]):
                e[:, h, 0] += scale * u * (np.abs(qs[h, :, 1:]) @ np.abs(k[h // group, :, 1:]).T).max(-1)
        bound = (u * (mag + size * (2 if r.vf == "q4_0" else 1)) + e * (size + mag)
                 + length * 2.0 ** -25 * np.abs(v).max())
        off = np.abs(np64(o[s:s + n]) - want)
        assert (off <= bound).all(), (b, float((off / bound).max()))


@pytest.mark.parametrize("step", [2.0, 12.0])
@pytest.mark.parametrize("n,kf,vf,dtype,D", RAMPS)
def test_frames_move_in_lone_tiles_and_pieces(fa, n, kf, vf, dtype, D, step):
    """Scores that grow by `step` a key block, past the 10-point margin in every block or in every sixth, in
    tiles alone in their unit (1 and 5 tokens) and in pairs, in units that stay whole (of up to 8 blocks) and
    in pieces of several blocks, which are then merged with frames far apart.  The launches give the same
    bytes.  (The largest score before scaling is below 2^13, so that its f32 accumulation over D / 16
    products of 16, each rounded within 2^-23, moves a scaled score by less than 8 * 2^-10 / 8 = 2^-10 at
    worst.)"""
    Hkv, page = 8, 128
    lens = [2500 + 37 * b for b in range(10 if n < 300 else 1)] + [900, 300 if n == 300 else 129]
    r = make_ragged([n] * len(lens), lens, Hkv, D, page, dtype, "dense", vf, seed=211, poison=False)
    for b, length in enumerate(lens):
        for p in range(-(-length // page)):
            r.k[int(r.table[b, p]), :, :, 0] = step * p / (8.0 * D ** -0.5)
    if kf == "q4_0":
        r.k, r.kf = q4_buffer(r.k), kf
    q = make_q(sum(r.new), 4 * Hkv, D, dtype, seed=212)
    q[..., 0] = 8.0
    o = run(fa, r, q)
    check_ramp(r, q, o.cpu())
    args = (q.cuda(), r.pool(fa, "k"), r.pool(fa, "v"), *r.batch())
    for _ in range(20):
        assert torch.equal(o, fa.fa_prefill_paged(*args))
    assert fa.fa_get_status() == fa.FA_OK


@pytest.mark.parametrize("D,kf,vf", [(128, "dense", "dense"), (64, "q4_0", "q4_0"), (128, "dense", "q4_0"),
                                     (128, "q4_0", "q4_0")])
def test_merged_rows_at_other_strides(fa, D, kf, vf):
    """Rows of cut units (two and many pieces) stored by the merges: o head-major, o with gaps between rows
    and heads; what lies between stays as it was."""
    new, Hq, Hkv, first, pad = [1, 600, 2, 77], 8, 2, 3, 6
    lens = [9000, 4000, 3001, 1500]
    n, rows = sum(new), first + sum(new) + pad
    r = make_ragged(new, lens, Hkv, D, 64, "f16", kf, vf, seed=221, first_row=first)
    fused = make_q(rows, Hq + 2 * Hkv, D, "f16", seed=222).cuda()
    q = fused[:, :Hq]
    k, v, batch = r.pool(fa, "k"), r.pool(fa, "v"), r.batch()
    want = fa.fa_prefill_paged(q.contiguous(), k, v, *batch)
    check(r, q.cpu(), want.cpu())
    whole = torch.full((Hq, rows, D), 7.0, dtype=torch.float16, device="cuda")
    gaps = torch.full((rows, Hq + 3, D + 8), 7.0, dtype=torch.float16, device="cuda")
    for o in (whole.transpose(0, 1), gaps[:, 1:Hq + 1, :D]):
        for _ in range(10):
            o[first:first + n] = 0
            fa.fa_prefill_paged(q, k, v, *batch, o)
            assert torch.equal(o[first:first + n], want[first:first + n])
        assert (o[:first] == 7.0).all() and (o[first + n:] == 7.0).all()
    assert fa.fa_get_status() == fa.FA_OK
    assert (gaps[:, 0] == 7.0).all() and (gaps[:, Hq + 1:] == 7.0).all() and (gaps[..., D:] == 7.0).all()


@pytest.mark.parametrize("D,kf,vf", [(128, "dense", "dense"), (64, "dense", "q4_0"), (128, "q4_0", "q4_0"),
                                     (64, "q4_0", "q4_0")])
def test_cut_units_without_the_causal_mask(fa, D, kf, vf):
    """All keys for every row: chunks and single tokens in many pieces, rows before the first key's position
    among them."""
    r = make_ragged([300, 1, 5, 40], [5000, 9000, 3, 1300], 2, D, 64, "f16", kf, vf, seed=231)
    q = make_q(sum(r.new), 8, D, "f16", seed=232)
    first = run(fa, r, q, causal=False)
    check(r, q, first.cpu(), causal=False)
    for _ in range(10):
        assert torch.equal(first, run(fa, r, q, causal=False))
