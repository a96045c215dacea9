"""Writing rows into page pools (fa_append_paged) and reading them back (fa_read_paged).  Both are
exact: q4_0 planes are compared bit for bit with the oracle's quantizer, dense pools and read values
with the only rounding the format allows ((nibble - 8) * scale, exact in f32, to the dtype)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import np64
from paged_common import DT, make_ragged, q4_buffer, q4_planes

pytestmark = pytest.mark.gpu


def places(r):
    """(packed row, page, slot) of every row of the batch."""
    page = r.shape[2]
    out = []
    for b, (n, length) in enumerate(zip(r.new, r.lens)):
        for i in range(n):
            pos = length - n + i
            out.append((int(r.starts[b]) + i, int(r.table[b, pos // page]), pos % page))
    return np.array(out, dtype=np.int64).reshape(-1, 3)


def after_append(r, side, x):
    """The pool (CPU, as stored) after x [rows, Hkv, D] has been written."""
    t, fmt = (r.k, r.kf) if side == "k" else (r.v, r.vf)
    row, page, slot = places(r).T
    t = t.clone()
    if fmt == "dense":
        t[page, :, slot] = x[row]
        return t
    nib, sc = oracle.quantize_q4_0(x[row][:, :, None].float().numpy())
    n, s = q4_planes(t, r.shape)
    n[page, :, slot] = torch.from_numpy(nib[:, :, 0])
    s[page, :, slot] = torch.from_numpy(sc[:, :, 0].view(np.int16).copy())
    return t


def stored(pool):
    """A pool's bits on the CPU."""
    t = pool if isinstance(pool, torch.Tensor) else pool.buf
    return t.cpu() if t.dtype == torch.uint8 else t.cpu().view(torch.int16)


def bits(t):
    return t if t.dtype == torch.uint8 else t.view(torch.int16)


def expected_read(r, side, rows):
    """{packed row: [Hkv, D]} in the dtype."""
    got = {}
    for b, (n, length) in enumerate(zip(r.new, r.lens)):
        if n:
            x = torch.from_numpy(r.sequence(side, b)[:, length - n:]).to(DT[r.dtype])
            for i in range(n):
                got[int(r.starts[b]) + i] = x[:, i]
    return got


CASES = [
    # new, lens, Hkv, D, page, dtype, kf, vf
    ([1], [1], 1, 32, 1, "f16", "dense", "dense"),
    ([1], [1], 1, 32, 1, "f16", "q4_0", "q4_0"),
    ([5, 0, 1, 40], [5, 9, 129, 200], 2, 128, 128, "f16", "q4_0", "q4_0"),
    ([5, 0, 1, 40], [70, 9, 1, 200], 8, 128, 16, "bf16", "dense", "dense"),
    ([17, 300, 2], [1000, 300, 77], 3, 64, 48, "bf16", "q4_0", "dense"),
    ([1] * 33, list(range(1, 34)), 4, 96, 7, "f16", "dense", "q4_0"),
    ([600, 1], [601, 4000], 8, 128, 256, "f16", "q4_0", "q4_0"),
    ([3, 2], [30, 2], 2, 576, 5, "bf16", "q4_0", "dense"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[2:])) + f"-B{len(c[0])}")
def test_append_and_read(fa, case):
    new, lens, Hkv, D, page, dtype, kf, vf = case
    r = make_ragged(new, lens, Hkv, D, page, dtype, kf, vf, seed=sum(lens))
    rows = sum(new)
    k_out = torch.empty(rows, Hkv, D, dtype=DT[dtype], device="cuda")
    v_out = torch.empty_like(k_out)
    fa.fa_read_paged(r.pool(fa, "k"), r.pool(fa, "v"), *r.batch(), k_out, v_out)
    for side, out in (("k", k_out), ("v", v_out)):
        want = expected_read(r, side, rows)
        for t, x in want.items():
            assert torch.equal(bits(out[t].cpu()), bits(x)), (side, t)
    g = torch.Generator().manual_seed(7)
    k_new, v_new = (torch.randn(rows, Hkv, D, generator=g).to(DT[dtype]) for _ in "kv")
    k, v = r.pool(fa, "k"), r.pool(fa, "v")
    fa.fa_append_paged(k_new.cuda(), v_new.cuda(), k, v, *r.batch())
    assert fa.fa_get_status() == fa.FA_OK
    # every byte of the pools: the rows' slots as the format defines them, all others untouched
    assert torch.equal(stored(k), bits(after_append(r, "k", k_new)))
    assert torch.equal(stored(v), bits(after_append(r, "v", v_new)))


def test_special_blocks(fa):
    """Zero blocks (scale -0), ties of the largest magnitude with either sign first, subnormals."""
    D = 64
    x = torch.zeros(6, 2, D, dtype=torch.float16)
    x[1, 0, 3], x[1, 0, 9] = -2.5, 2.5
    x[2, 0, 3], x[2, 0, 9] = 2.5, -2.5
    x[3] = 6e-8
    x[4, :, ::2] = 65504.0
    x[5] = torch.linspace(-1, 1, D)
    r = make_ragged([6], [9], 2, D, 4, "f16", "q4_0", "q4_0", seed=1)
    k, v = r.pool(fa, "k"), r.pool(fa, "v")
    fa.fa_append_paged(x.cuda(), x.flip(0).cuda(), k, v, *r.batch())
    assert torch.equal(stored(k), after_append(r, "k", x))
    assert torch.equal(stored(v), after_append(r, "v", x.flip(0)))


def test_strides_padding_and_one_side(fa):
    """Rows cut out of a fused projection, a broadcast value row, head-major outputs, rows before the
    first sequence and behind the last one, and K alone."""
    new, lens, Hkv, D, page, first, pad = [20, 1, 9], [50, 300, 9], 2, 128, 16, 2, 5
    rows = first + sum(new) + pad
    for fmt in ("dense", "q4_0"):
        r = make_ragged(new, lens, Hkv, D, page, "f16", fmt, fmt, seed=5, first_row=first)
        fused = torch.randn(rows, 4 + 2 * Hkv, D, generator=torch.Generator().manual_seed(2)).half()
        fg = fused.cuda()
        k, v = r.pool(fa, "k"), r.pool(fa, "v")
        one = fg[:1, 4 + Hkv:].expand(rows, Hkv, D)
        fa.fa_append_paged(fg[:, 4:4 + Hkv], one, k, v, *r.batch())
        wk = after_append(r, "k", fused[:, 4:4 + Hkv])
        wv = after_append(r, "v", fused[:1, 4 + Hkv:].expand(rows, Hkv, D))
        assert torch.equal(stored(k), bits(wk)) and torch.equal(stored(v), bits(wv))
        k1 = r.pool(fa, "k")
        fa.fa_append_paged(fg[:, 4:4 + Hkv], None, k1, None, *r.batch())
        assert torch.equal(stored(k1), bits(wk))
        r.k, r.v = wk, wv
        out = torch.full((Hkv, rows, D), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
        got, none = fa.fa_read_paged(k, None, *r.batch(), out)
        assert got is out and none is None
        for t, x in expected_read(r, "k", rows).items():
            assert torch.equal(bits(out[t].cpu().contiguous()), bits(x.contiguous()))
        assert (out[:first] == 7.0).all() and (out[rows - pad:] == 7.0).all()
        assert fa.fa_get_status() == fa.FA_OK


def test_many_sequences(fa):
    """More sequences than the kernels keep in shared memory, many of them empty."""
    rng = np.random.default_rng(3)
    B = 1500
    new = [int(x) for x in rng.integers(0, 3, B)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 9, B))]
    r = make_ragged(new, lens, 1, 64, 4, "bf16", "q4_0", "dense", seed=9)
    g = torch.Generator().manual_seed(7)
    k_new, v_new = (torch.randn(sum(new), 1, 64, generator=g).bfloat16() for _ in "kv")
    k, v = r.pool(fa, "k"), r.pool(fa, "v")
    fa.fa_append_paged(k_new.cuda(), v_new.cuda(), k, v, *r.batch())
    assert torch.equal(stored(k), bits(after_append(r, "k", k_new)))
    assert torch.equal(stored(v), bits(after_append(r, "v", v_new)))
    out = torch.empty(sum(new), 1, 64, dtype=torch.bfloat16, device="cuda")
    fa.fa_read_paged(v, None, *r.batch(), out)
    assert torch.equal(bits(out.cpu()), bits(v_new))
    assert fa.fa_get_status() == fa.FA_OK


@pytest.mark.parametrize("fmt", ["dense", "q4_0"])
def test_bad_batches_are_reported_and_skipped(fa, fmt):
    Hkv, D, page = 2, 64, 8
    r = make_ragged([4, 3], [20, 11], Hkv, D, page, "f16", fmt, fmt, seed=2)
    x = torch.randn(7, Hkv, D, generator=torch.Generator().manual_seed(7)).half()
    table, starts, lens = r.batch()
    before = stored(r.pool(fa, "k"))

    def call(table, starts, lens):
        k, v = r.pool(fa, "k"), r.pool(fa, "v")
        out = torch.full((7, Hkv, D), 7.0, dtype=torch.float16, device="cuda")
        fa.fa_append_paged(x.cuda(), x.cuda(), k, v, table, starts, lens)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        fa.fa_read_paged(k, None, table, starts, lens, out)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        return stored(k), out

    for bad in ([0, 5, 4], [-1, 4, 7], [0, 4, 8]):
        k, out = call(table, torch.tensor(bad, dtype=torch.int32, device="cuda"), lens)
        assert torch.equal(k, before) and (out == 7.0).all()
    # the second sequence alone is written and read
    only = make_ragged([4, 3], [20, 11], Hkv, D, page, "f16", fmt, fmt, seed=2)
    only.new = [0, 3]
    only.starts = torch.tensor([4, 4, 7], dtype=torch.int32)
    want = bits(after_append(only, "k", x))
    for t0, n0 in ((r.shape[0], 20), (-1, 20), (None, 25), (None, -3)):
        t, l_ = table.clone(), lens.clone()
        if t0 is not None:
            t[0, 2] = t0  # the page of positions 16 .. 19
        l_[0] = n0 if t0 is not None or n0 < 0 else 8 * table.shape[1] + 1
        k, out = call(t, starts, l_)
        assert torch.equal(k, want)
        assert (out[:4] == 7.0).all() and (out[4:] != 7.0).any()
    # more rows than tokens: the rows at positions below 0 are skipped
    k, out = call(table, starts, torch.tensor([20, 2], dtype=torch.int32, device="cuda"))
    assert (out[4] == 7.0).all() and (out[5:] != 7.0).any()


def test_captured_append_attend_read(fa):
    """A serving step as it is used: append, attend, decode and read in one captured graph, replayed
    step by step as the sequences grow, against the oracle on the tokens written so far."""
    from test_gpu_prefill_paged import check, make_q

    Hq, Hkv, D, page, B, rows = 8, 2, 128, 128, 3, 40
    pools = torch.zeros(8, Hkv, page, D).half()
    k = fa.Q4Tensor(q4_buffer(pools).cuda(), *pools.shape)
    v = pools.clone().cuda()
    table = torch.tensor([[3, 1], [0, 6], [7, 2]], dtype=torch.int32)
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(rows, Hq, D, dtype=torch.float16, device="cuda")
    kn, vn = (torch.zeros(rows, Hkv, D, dtype=torch.float16, device="cuda") for _ in "kv")
    o, k_out, v_out = torch.zeros_like(q), torch.zeros_like(kn), torch.zeros_like(vn)
    ws = torch.empty(fa.fa_prefill_paged_workspace_bytes(Hq, Hkv, D), dtype=torch.uint8,
                     device="cuda")
    tab = table.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_append_paged(kn, vn, k, v, tab, starts, lens)
        fa.fa_prefill_paged(q, k, v, tab, starts, lens, o, workspace=ws)
        fa.fa_read_paged(k, v, tab, starts, lens, k_out, v_out)
    have = [0] * B
    for step, new in enumerate(([30, 9, 1], [1, 1, 1], [1, 38, 1], [1, 1, 1], [0, 1, 20])):
        have = [h + n for h, n in zip(have, new)]
        x = make_q(rows, Hq + 2 * Hkv, D, "f16", seed=200 + step)
        q.copy_(x[:, :Hq])
        kn.copy_(x[:, Hq:Hq + Hkv])
        vn.copy_(x[:, Hq + Hkv:])
        st = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32)
        starts.copy_(st)
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        g.replay()
        assert fa.fa_get_status() == fa.FA_OK
        r = make_ragged(new, have, Hkv, D, page, "f16", "q4_0", "dense", seed=0)
        r.shape, r.table, r.starts = tuple(pools.shape), table, st
        r.k, r.v = k.buf.cpu(), v.cpu()
        check(r, q.cpu(), o.cpu())
        n = sum(new)
        assert torch.equal(v_out[:n], vn[:n])
        nib, sc = oracle.quantize_q4_0(kn[:n, :, None].cpu().float().numpy())
        want = torch.from_numpy(oracle.dequantize_q4_0(nib, sc)[:, :, 0]).half()
        assert torch.equal(k_out[:n].cpu(), want)
        if new == [1, 1, 1]:
            d = fa.fa_decode_paged(q[:3, :, None].contiguous(), k, v, tab, lens)
            assert fa.fa_get_status() == fa.FA_OK
            check(r, q.cpu(), d[:, :, 0].cpu())


def test_read_is_exact_at_the_values_bounds(fa):
    """Every nibble against the largest, smallest and subnormal scales, both dtypes."""
    D, page = 32, 4
    for dtype in ("f16", "bf16"):
        shape = (2, 1, page, D)
        r = make_ragged([8], [8], 1, D, page, dtype, "q4_0", "q4_0", seed=1, spare=0)
        nib, sc = q4_planes(r.k, shape)
        nib[:] = torch.arange(16, dtype=torch.uint8) | (torch.arange(16, dtype=torch.uint8) << 4)
        sc[:] = torch.tensor([0x7BFF - (1 << 12), 0x0001, 0x03FF, -0x8000 + 1, 0x3C00, 0x2E66, 0,
                              -0x8000], dtype=torch.int32).to(torch.int16).view(2, 1, page, 1)
        out = torch.empty(8, 1, D, dtype=DT[dtype], device="cuda")
        fa.fa_read_paged(r.pool(fa, "k"), None, *r.batch(), out)
        for t, x in expected_read(r, "k", 8).items():
            assert torch.equal(out[t].cpu(), x), (dtype, t)
        assert np.isfinite(np64(out)).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_value_quantizes_as_in_the_contiguous_call(fa, dtype):
    """All 2^16 bit patterns (infinities and NaN among them), in order and shuffled, and blocks of few
    distinct magnitudes, whose largest recurs in any lane with either sign: the bits that the
    contiguous quantizer stores."""
    D, page = 128, 64
    g = torch.Generator().manual_seed(11)
    every = torch.arange(65536, dtype=torch.int32)
    few = torch.tensor([-3.0, -1.5, 0.0, 1.5, 3.0]).to(DT[dtype])
    x = torch.cat([every.to(torch.int16), every[torch.randperm(65536, generator=g)].to(torch.int16),
                   few[torch.randint(5, (65536,), generator=g)].view(torch.int16)])
    x = x.view(DT[dtype]).reshape(-1, 1, D).cuda()
    rows = x.shape[0]
    assert rows % page == 0
    want = fa.fa_quantize_q4_0(x.reshape(1, 1, rows, D))
    pools = [fa.Q4Tensor(torch.zeros_like(want.buf), rows // page, 1, page, D) for _ in "kv"]
    table = torch.arange(rows // page, dtype=torch.int32, device="cuda")[None]
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    lens = torch.tensor([rows], dtype=torch.int32, device="cuda")
    fa.fa_append_paged(x, x, *pools, table, starts, lens)
    assert fa.fa_get_status() == fa.FA_OK
    n = rows * D // 2
    for p in pools:
        assert torch.equal(p.buf[:n], want.buf[:n])
        assert torch.equal(p.buf[-rows * D // 16:], want.buf[-rows * D // 16:])


@pytest.mark.parametrize("Hkv,D,rows", [(1, 128, 5003), (1, 64, 9001), (5, 64, 700), (5, 128, 3001),
                                        (3, 160, 1777), (40, 32, 333), (7, 256, 211), (64, 128, 5)])
def test_rows_and_heads_split_over_ctas(fa, Hkv, D, rows):
    """Several groups of rows per CTA, part of the heads per CTA, the last of each short."""
    new, lens = [rows - 2 * (rows // 3), 0, 2 * (rows // 3)], [rows, 3, rows]
    r = make_ragged(new, lens, Hkv, D, 32, "f16", "q4_0", "dense", seed=rows)
    k_out = torch.empty(rows, Hkv, D, dtype=torch.float16, device="cuda")
    v_out = torch.empty_like(k_out)
    fa.fa_read_paged(r.pool(fa, "k"), r.pool(fa, "v"), *r.batch(), k_out, v_out)
    for side, out in (("k", k_out), ("v", v_out)):
        want = expected_read(r, side, rows)
        assert torch.equal(bits(out.cpu()), bits(torch.stack([want[t] for t in range(rows)])))
    g = torch.Generator().manual_seed(12)
    k_new, v_new = (torch.randn(rows, Hkv, D, generator=g).half() for _ in "kv")
    k, v = r.pool(fa, "k"), r.pool(fa, "v")
    fa.fa_append_paged(k_new.cuda(), v_new.cuda(), k, v, *r.batch())
    assert fa.fa_get_status() == fa.FA_OK
    assert torch.equal(stored(k), bits(after_append(r, "k", k_new)))
    assert torch.equal(stored(v), bits(after_append(r, "v", v_new)))


@pytest.mark.parametrize("fmt", ["dense", "q4_0"])
def test_lengths_at_the_ends_of_32_bits(fa, fmt):
    """Every length that the table cannot hold is reported and its rows skipped, down to -2^31, from
    which a row's place is no longer a difference of 32 bits; the other sequence is written and read."""
    Hkv, D, page = 2, 64, 8
    r = make_ragged([4, 3], [20, 11], Hkv, D, page, "f16", fmt, fmt, seed=2)
    x = torch.randn(7, Hkv, D, generator=torch.Generator().manual_seed(7)).half()
    table, starts, _ = r.batch()
    only = make_ragged([4, 3], [20, 11], Hkv, D, page, "f16", fmt, fmt, seed=2)
    only.new = [0, 3]
    only.starts = torch.tensor([4, 4, 7], dtype=torch.int32)
    want = bits(after_append(only, "k", x))
    for n in (-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 3, -2 ** 31 + 4, -1, 2 ** 31 - 1, 2 ** 30):
        lens = torch.tensor([n, 11], dtype=torch.int32, device="cuda")
        k, v = r.pool(fa, "k"), r.pool(fa, "v")
        out = torch.full((7, Hkv, D), 7.0, dtype=torch.float16, device="cuda")
        fa.fa_append_paged(x.cuda(), x.cuda(), k, v, table, starts, lens)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        fa.fa_read_paged(k, None, table, starts, lens, out)
        assert fa.fa_get_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(stored(k), want), n
        assert (out[:4] == 7.0).all() and (out[4:] != 7.0).any()


@pytest.mark.parametrize("B", [3, 1500])
def test_bad_length_of_a_sequence_without_rows_is_reported(fa, B):
    """In a batch that fits shared memory and in a larger one; the rows of the others are moved."""
    Hkv, D, page = 1, 64, 16
    pool = torch.zeros(4, Hkv, page, D, dtype=torch.float16, device="cuda")
    x = torch.randn(2, Hkv, D, generator=torch.Generator().manual_seed(8)).half().cuda()
    table = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    table[0], table[B - 1] = torch.tensor([1, 2]), torch.tensor([3, 0])
    starts = torch.ones(B + 1, dtype=torch.int32, device="cuda")
    starts[0], starts[B] = 0, 2
    for n in (0, 33, -1, -2 ** 31):
        lens = torch.full((B,), 32, dtype=torch.int32, device="cuda")
        lens[B // 2] = n
        status = fa.FA_OK if n == 0 else fa.FA_ERR_INVALID_ARG
        out = torch.empty_like(x)
        fa.fa_append_paged(x, None, pool, None, table, starts, lens)
        assert fa.fa_get_status() == status
        fa.fa_read_paged(pool, None, table, starts, lens, out)
        assert fa.fa_get_status() == status
        assert torch.equal(out, x)
