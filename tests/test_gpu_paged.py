"""The paged latent cache on the GPU against its float64 form: ragged batches, pages that end inside a tile, NaN in
every row that must not matter, padded batches, lists of blocks, captured and replayed steps."""
import concurrent.futures
import math
import threading

import pytest
import torch

from mla_latent_kv_31_b200 import mla, synth
from paged_testlib import DT, HALF, NAN, Case, handle, rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    m = {dt: handle(dt) for dt in ("bf16", "fp32")}
    yield m
    for x in m.values():
        x.close()


def ok(m):
    s = m.sync_status()
    assert s == 0, (mla.mla_status_string(s), hex(mla.mla_device_error_bits(m.handle)))


def flagged(m, bit):
    assert m.sync_status() == 7
    assert mla.mla_device_error_bits(m.handle) == bit


def prefix(c):
    return lambda t, b, pos: c.rows[b][:pos + 1]


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("dtype,page,lens,tq", [
    ("fp32", 16, LENS, [1] * 14), ("fp32", 32, [40, 700, 3, 129], [5, 1, 3, 0]), ("fp32", 48, [1000], [130]),
    ("bf16", 16, LENS, [1] * 14), ("bf16", 64, LENS, [1] * 14), ("bf16", 32, [40, 700, 3, 129], [5, 1, 3, 0]),
    ("bf16", 48, [200, 1000, 47], [3, 2, 1]), ("bf16", 80, [321, 79, 81, 400], [2, 2, 2, 2]),
    ("bf16", 128, [1025, 128, 5], [1, 8, 5]), ("bf16", 192, [700, 191], [1, 4]),
    ("bf16", 64, [4097], [1]), ("bf16", 64, [9000, 77], [1, 1]), ("bf16", 64, [300], [300]),
    ("bf16", 1024, [1500, 2049], [2, 1]), ("bf16", 64, [300, 700, 512, 513, 1000] * 11, [1] * 55),
    ("bf16", 64, [257, 900, 600, 5, 1025] * 3, [1, 0, 1, 1, 1] * 3)])
def test_attention(mods, dtype, page, lens, tq):
    c = Case(dtype, page, lens, tq, seed=len(lens) + page)
    o, lse = mods[dtype].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods[dtype])
    c.check_attention(o, lse, prefix(c))


@pytest.mark.parametrize("B,n,hi,pad", [(2, 2, 700, 0), (9, 2, 2500, 3), (40, 2, 300, 0), (7, 3, 900, 1), (3, 5, 1300, 0),
                                        (13, 7, 400, 2), (4, 16, 700, 0), (5, 14, 333, 0), (2, 11, 5000, 0),
                                        (3, 64, 300, 5), (2, 74, 200, 0)])
def test_attention_even_batches(mods, B, n, hi, pad):
    """The same number of new tokens everywhere, lengths from none behind them to hi: the walk's other orders."""
    c = Case("bf16", 16, [n + (hi - n) * b // max(B - 1, 1) for b in range(B)], [n] * B, seed=62 + n, pad=pad)
    o, lse = (torch.full((c.T + pad, 128, *w), 7.0, dtype=dt, device="cuda")
              for w, dt in (((512,), torch.bfloat16), ((), torch.float32)))
    mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope, o, lse)
    ok(mods["bf16"])
    c.check_attention(o, lse, prefix(c))
    assert (o[c.T:] == 7).all() and (lse[c.T:] == 7).all()
    c.d_lens[1] = n - 1                                    # fewer rows than new tokens
    mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope, o, lse)
    flagged(mods["bf16"], 1 << 1)
    assert (o[n:2 * n] == 0).all() and torch.isneginf(lse[n:2 * n]).all()
    tokens = c.tokens()
    c.tokens = lambda: [x for x in tokens if x[1] != 1]
    c.check_attention(o, lse, prefix(c))


def test_attention_uneven_chunks_of_many_tokens(mods):
    """Two to four tokens a pair of CTAs, sequences of 0 to 64 new tokens, one of them flagged."""
    tq = [50, 0, 64, 1, 33, 7, 40, 20]
    c = Case("bf16", 32, [300, 40, 64, 500, 33, 600, 41, 290], tq, seed=63, pad=2)
    c.d_lens[6] = 39                                       # fewer rows than new tokens
    o, lse = mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope)
    flagged(mods["bf16"], 1 << 1)
    a, b = int(c.cu[6]), int(c.cu[7])
    assert (o[a:b] == 0).all() and torch.isneginf(lse[a:b]).all()
    tokens = [x for x in c.tokens() if x[1] != 6]
    c.tokens = lambda: tokens
    c.check_attention(o, lse, prefix(c))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_many_short_sequences(mods, dtype):
    c = Case(dtype, 16, [1 + 7 * i % 90 for i in range(200)], [1] * 200, seed=3)
    o, lse = mods[dtype].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods[dtype])
    c.check_attention(o, lse, prefix(c))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_padded_batch_and_strided_table(mods, dtype):
    c = Case(dtype, 64, [130, 64, 700], [2, 0, 3], pad=6, seed=4)
    wide = torch.full((3, c.table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.d_table
    b = mla.PagedBatch(c.cache, wide[:, :c.table.shape[1]], c.d_cu, c.d_lens, c.T + 6)
    o = torch.full((c.T + 6, c.dims.n_h, c.dims.d_c), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((c.T + 6, c.dims.n_h), 7.0, device="cuda")
    mods[dtype].attn_paged(b, c.q_abs, c.q_rope, o, lse)
    ok(mods[dtype])
    c.check_attention(o, lse, prefix(c))
    assert (o[c.T:] == 7).all() and (lse[c.T:] == 7).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_later_rows_may_be_nan(mods, dtype):
    """The last two rows of the sequence are NaN: the tokens before them do not see it."""
    c = Case(dtype, 16, [70], [5], seed=5)
    for p in (68, 69):
        c.cache[c.table[0, p // 16].long(), p % 16] = NAN
    o, lse = mods[dtype].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods[dtype])
    assert torch.isnan(o[3:]).any()
    c.tq, c.lens = [3], [68]                              # the first three tokens alone
    c.check_attention(o, lse, prefix(c))


def test_attention_shared_prefix_pages(mods):
    c = Case("bf16", 32, [200, 170, 96 + 5], [1, 2, 4], seed=6, share=3)
    o, lse = mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods["bf16"])
    c.check_attention(o, lse, prefix(c))


def test_attention_large_scores(mods):
    """Rows whose scores rise by hundreds along the sequence: the running maximum moves at every tile."""
    c = Case("bf16", 64, [1000], [1], seed=7)
    r = c.rows[0]
    d = c.dims.d_c
    r[:, :d] = c.q[0, 0, :d] * torch.linspace(0.0, 40.0, 1000, dtype=torch.float64)[:, None]
    r[:] = r.to(torch.bfloat16).double()
    pos = torch.arange(1000)
    c.cache[c.table[0, pos // 64].long().cuda(), (pos % 64).cuda()] = r.to(torch.bfloat16).cuda()
    o, lse = mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods["bf16"])
    c.check_attention(o, lse, prefix(c))


@pytest.mark.parametrize("dtype,page,lens,tq,low", [("fp32", 16, [300, 140, 139], [2, 1, 3], 140),
                                                    ("bf16", 64, [700, 300, 256], [2, 1, 3], 300),
                                                    ("bf16", 64, [5000, 20], [1, 1], 1500)])
def test_attention_scores_of_minus_infinity(mods, dtype, page, lens, tq, low):
    """The first `low` rows of each sequence score -inf: weights of 0; where no other row is seen, an empty row."""
    c = Case(dtype, page, lens, tq, seed=67)
    d = c.dims.d_c
    c.q[..., d] = -c.q[..., d].abs() - 0.5
    for b, n in enumerate(lens):
        j = torch.arange(min(low, n))
        c.cache[c.table[b, j // page].long().cuda(), (j % page).cuda(), d] = float("inf")
    o, lse = mods[dtype].attn_paged(c.batch(), c.q_abs, c.q_rope)
    blocks = torch.full((c.T, max(lens) // page + 1), -1, dtype=torch.int32)
    for t, b, pos in c.tokens():
        blocks[t, :pos // page + 1] = torch.arange(pos // page + 1, dtype=torch.int32)
    o2, lse2 = mods[dtype].attn_paged_sparse(c.batch(), c.q_abs, c.q_rope, blocks.cuda())
    ok(mods[dtype])
    for x, y in ((o, lse), (o2, lse2)):
        c.check_attention(x, y, lambda t, b, pos: c.rows[b][low:pos + 1])


@pytest.mark.parametrize("dtype,lens", [("fp32", [700, 40]), ("bf16", [5000, 40]), ("bf16", [200, 40]),
                                        ("bf16", [256 * 74 * 2, 300])])
def test_attention_carries_nan_to_its_heads_and_tokens(mods, dtype, lens):
    """A NaN in a query makes all scores of its head NaN, NaN rows those of a part of a token's keys: the output is NaN
    there, in however many pieces the token is dealt, and the other heads and tokens keep their values bit for bit."""
    m = mods[dtype]
    c = Case(dtype, 16, lens, [1, 1], seed=68)
    qa, qr, b = c.q_abs, c.q_rope, c.batch()
    o, lse = m.attn_paged(b, qa, qr)
    bad = qa.clone()
    bad[0, 2, 3] = NAN
    o2, lse2 = m.attn_paged(b, bad, qr)
    ok(m)
    assert torch.isnan(o2[0, 2]).all() and torch.isnan(lse2[0, 2])
    o2[0, 2], lse2[0, 2] = o[0, 2], lse[0, 2]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    j = torch.arange(lens[0] // 3)
    c.cache[c.table[0, j // 16].long().cuda(), (j % 16).cuda()] = NAN
    o2, lse2 = m.attn_paged(b, qa, qr)
    ok(m)
    assert torch.isnan(o2[0]).all() and torch.isnan(lse2[0]).all()
    assert torch.equal(o[1], o2[1]) and torch.equal(lse[1], lse2[1])


def test_attention_equals_the_contiguous_core(mods):
    c = Case("bf16", 64, [500, 1, 129], [1, 1, 1], seed=8)
    o, lse = mods["bf16"].attn_paged(c.batch(), c.q_abs, c.q_rope)
    rows = torch.cat(c.rows).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 500, 501, 630], dtype=torch.int64, device="cuda")
    o2, lse2 = mods["bf16"].attn_decode_latent(c.q_abs, c.q_rope, 3, 1, cu, rows)
    ok(mods["bf16"])
    # each side is within 2 * 2^-8 of sum p |c| (weights and output or partial rounded to bf16)
    lim = 4 * HALF["bf16"] * max(float(r[:, :512].abs().max()) for r in c.rows)
    assert (o.float() - o2).abs().max() <= lim
    assert (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_is_deterministic_and_runs_on_any_stream(mods, dtype):
    m = mods[dtype]
    c = Case(dtype, 64, [700, 64, 3000], [2, 1, 1], seed=9)
    b, qa, qr = c.batch(), c.q_abs, c.q_rope
    o, lse = m.attn_paged(b, qa, qr)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, lse2 = m.attn_paged(b, qa, qr)
    torch.cuda.synchronize()
    ok(m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_calls_take_every_name_of_their_device(mods):
    m = mods["bf16"]
    c = Case("bf16", 64, [700, 64], [2, 1], seed=69)
    b, qa, qr = c.batch(), c.q_abs, c.q_rope
    o, lse = m.attn_paged(b, qa, qr)
    n = mla.mla_attn_paged_workspace(m.handle, 2, 3)
    torch.cuda.synchronize()
    for device in (0, "cuda:0", torch.device("cuda", 0), torch.device("cuda"), None):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            o2, lse2, ws = torch.zeros_like(o), torch.zeros_like(lse), torch.empty(n, dtype=torch.uint8, device="cuda")
            mla.mla_attn_paged(m.handle, b, qa, qr, o2, lse2, ws, n, device=device)
        assert mla.mla_sync_status(m.handle, s, device=device) == 0
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def in_fresh_thread(f):
    """f() in a thread that has made no CUDA call before."""
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        return pool.submit(f).result()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_calls_from_a_thread_without_cuda_calls_before(mods, dtype):
    """A handle that is ready, and a thread in which the call is the first to need the device's context."""
    m = mods[dtype]
    c = Case(dtype, 16, [700, 64], [2, 1], seed=72)
    d, b, qa, qr, kv = c.dims, c.batch(), c.q_abs, c.q_rope, c.on(c.normal(c.T, c.W))
    sums = c.summaries(c.normal(c.num_pages, c.W)).cuda()
    o, lse, out, blocks = torch.empty_like(qa), torch.empty(c.T, d.n_h, device="cuda"), torch.empty_like(qr), \
        torch.empty(c.T, 6, dtype=torch.int32, device="cuda")
    n = max(mla.mla_attn_paged_workspace(m.handle, 2, 3), mla.mla_paged_select_workspace(m.handle, 3, b.max_pages))
    ws, stream = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.cuda.current_stream().cuda_stream
    calls = [lambda: mla.mla_paged_append(m.handle, b, kv, c.W, qr, out, sums, stream),
             lambda: mla.mla_paged_select(m.handle, b, qa, qr, sums, 6, 1, 1, blocks, ws, n, stream),
             lambda: mla.mla_attn_paged_sparse(m.handle, b, qa, qr, blocks, 6, o, lse, ws, n, stream),
             lambda: mla.mla_attn_paged(m.handle, b, qa, qr, o, lse, ws, n, stream)]
    for call in calls:
        call()
        ok(m)
        outs = {0: [out], 1: [blocks], 2: [o, lse], 3: [o, lse]}[calls.index(call)]
        want = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        in_fresh_thread(call)
        ok(m)
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_layer_calls_from_a_thread_without_cuda_calls_before():
    """The same for the layer's append and decode, whose first step is a projection."""
    d, g = synth.V3, torch.Generator(device="cuda").manual_seed(73)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

    w = {"w_dq": normal(d.d_cq, d.d), "w_uq": normal(d.n_h * d.d_h, d.d_cq), "w_qr": normal(d.n_h * d.d_r, d.d_cq),
         "w_dkv": normal(d.d_c, d.d), "w_kr": normal(d.d_r, d.d), "w_uk": normal(d.n_h * d.d_h, d.d_c),
         "w_uv": normal(d.n_h * d.d_h, d.d_c), "w_o": normal(d.d, d.n_h * d.d_h)}
    m = mla.MLA(d, w)
    stream = torch.cuda.current_stream().cuda_stream
    h, cache, u = normal(2, d.d) * d.d ** 0.5, torch.zeros(2, d.d_c + d.d_r, dtype=torch.bfloat16, device="cuda"), normal(2, d.d)
    at = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.arange(2, device="cuda")
    cu = torch.tensor([0, 1, 2], device="cuda")
    na, nd = mla.mla_workspace_size(m.handle, mla.OP_CACHE_APPEND, 0, 1, 2), mla.mla_workspace_size(m.handle, mla.OP_DECODE, 2, 1)
    ws = torch.empty(max(na, nd), dtype=torch.uint8, device="cuda")
    calls = [(lambda: mla.mla_cache_append(m.handle, h, *at, 2, cache, 2, ws, na, stream), cache),
             (lambda: mla.mla_decode(m.handle, h, 2, 1, cu, cache, 2, u, ws, nd, stream), u)]
    for call, out in calls:
        call()
        ok(m)
        want = out.clone()
        out.zero_()
        in_fresh_thread(call)
        ok(m)
        assert torch.equal(out, want)
    m.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_first_calls_of_a_handle_from_several_threads(dtype):
    """Threads that make a handle's first calls at once, each on a stream of its own: as when they come one by one."""
    cases = [Case(dtype, 16, [300 + 90 * k, 20], [2, 1], seed=80 + k) for k in range(6)]
    jobs = [(c.batch(), c.q_abs, c.q_rope, c.summaries(c.normal(c.num_pages, c.W)).cuda(), torch.cuda.Stream()) for c in cases]

    def run(m, b, qa, qr, sums, s):
        with torch.cuda.stream(s):
            blocks = m.paged_select(b, qa, qr, sums, 6, 1, 1)
            return blocks, *m.attn_paged_sparse(b, qa, qr, blocks), *m.attn_paged(b, qa, qr)

    torch.cuda.synchronize()
    one, all_at_once = handle(dtype), handle(dtype)
    want = [run(one, *job) for job in jobs]
    ok(one)
    gate = threading.Barrier(len(jobs))
    with concurrent.futures.ThreadPoolExecutor(len(jobs)) as pool:
        got = list(pool.map(lambda job: (gate.wait(), run(all_at_once, *job))[1], jobs))
    torch.cuda.synchronize()
    ok(all_at_once)
    for x, y in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    one.close()
    all_at_once.close()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_runs(mods):
    """Queries of the attention core, then codes of the block scores, that are never loaded: every role gives up, the
    status says so, and the same call gives its usual results afterwards."""
    m = mods["bf16"]
    c = Case("bf16", 16, [3000, 700, 40], [2, 1, 3], seed=71)
    b, qa, qr, sums = c.batch(), c.q_abs, c.q_rope, c.summaries(c.normal(c.num_pages, c.W)).cuda()
    blocks = m.paged_select(b, qa, qr, sums, 8, 1, 1)
    calls = [lambda: m.attn_paged(b, qa, qr), lambda: m.attn_paged_sparse(b, qa, qr, blocks),
             lambda: (m.paged_select(b, qa, qr, sums, 8, 1, 1),)]
    for call in calls:
        want = [x.clone() for x in call()]
        ok(m)
        mla.mla_test_arm_paged_stall()
        call()
        assert m.sync_status() == 6 and mla.mla_device_error_bits(m.handle) == 1 << 6
        got = call()
        ok(m)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_flagged_batches_give_empty_rows(mods, dtype):
    m = mods[dtype]

    def run(c, batch):
        o, lse = m.attn_paged(batch, c.q_abs, c.q_rope)
        return o, lse

    c = Case(dtype, 32, [40, 70], [1, 2], seed=10)
    c.d_lens[1] = 1                                        # fewer rows than new tokens
    o, lse = run(c, c.batch())
    flagged(m, 1 << 1)
    assert (o[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    c.tq, c.lens = [1], [40]
    c.check_attention(o, lse, prefix(c))
    c = Case(dtype, 32, [40, 70], [1, 2], seed=10)
    c.d_lens[1] = 32 * c.table.shape[1] + 1                # longer than its table
    o, lse = run(c, c.batch())
    flagged(m, 1 << 7)
    assert (o[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    c = Case(dtype, 32, [40, 70], [1, 2], seed=10)
    c.d_cu[2] = 9                                          # past the rows given
    o, lse = run(c, c.batch())
    assert m.sync_status() == 7 and mla.mla_device_error_bits(m.handle) & (1 << 5)
    for bad in (c.num_pages, -1, 2 ** 31 - 1, -2 ** 31):
        c = Case(dtype, 32, [70, 40], [1, 1], seed=10)
        c.d_table[0, 1] = bad                              # rows 32 .. 63 are read as zeros
        o, lse = run(c, c.batch())
        flagged(m, 1 << 7)
        c.rows[0][32:64] = 0
        c.check_attention(o, lse, prefix(c))


# ---- chosen blocks ----------------------------------------------------------------------------------------
def listed_rows(c, blocks):
    def rows(t, b, pos):
        g = [x for x in blocks[t].tolist() if x >= 0]
        j = [x * c.page + k for x in g for k in range(c.page) if x * c.page + k <= pos]
        return c.rows[b][j]
    return rows


def random_blocks(c, top_k, seed, own=True):
    g = torch.Generator().manual_seed(seed)
    out = torch.full((c.T + c.pad, top_k), -1, dtype=torch.int32)
    for t, b, pos in c.tokens():
        nb = pos // c.page + 1
        n = min(nb, int(torch.randint(1, top_k + 1, (1,), generator=g)))
        pick = torch.randperm(nb, generator=g)[:n].tolist()
        if own and nb - 1 not in pick:
            pick[-1] = nb - 1
        out[t, :n] = torch.tensor(sorted(pick), dtype=torch.int32)
    return out


@pytest.mark.parametrize("dtype,page,lens,tq,top_k", [
    ("fp32", 16, [300, 40, 1, 17], [5, 2, 1, 1], 6), ("bf16", 16, [300, 40, 1, 17], [5, 2, 1, 1], 20),
    ("bf16", 64, [3000, 100, 64], [9, 1, 3], 12), ("bf16", 128, [2000], [40], 5), ("bf16", 48, [500, 95], [2, 2], 7)])
@pytest.mark.parametrize("own", [True, False])
def test_sparse_attention(mods, dtype, page, lens, tq, top_k, own):
    c = Case(dtype, page, lens, tq, seed=page + top_k)
    blocks = random_blocks(c, top_k, 1, own)
    blocks[0] = -1                                         # a token that attends to nothing
    o, lse = mods[dtype].attn_paged_sparse(c.batch(), c.q_abs, c.q_rope, blocks.cuda())
    ok(mods[dtype])
    c.check_attention(o, lse, listed_rows(c, blocks))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sparse_over_all_blocks_is_the_whole_attention(mods, dtype):
    c = Case(dtype, 64, [777, 130], [3, 2], seed=11)
    blocks = torch.full((c.T, 13), -1, dtype=torch.int32)
    for t, b, pos in c.tokens():
        blocks[t, :pos // 64 + 1] = torch.arange(pos // 64 + 1, dtype=torch.int32)
    o, lse = mods[dtype].attn_paged_sparse(c.batch(), c.q_abs, c.q_rope, blocks.cuda())
    o2, lse2 = mods[dtype].attn_paged(c.batch(), c.q_abs, c.q_rope)
    ok(mods[dtype])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [[3, 3, 4], [2, 1, 4], [0, 1, 5], [0, 1, 2 ** 31 - 1]])
def test_sparse_flags_lists_that_do_not_ascend(mods, dtype, bad):
    c = Case(dtype, 16, [70, 70], [1, 1], seed=12)         # own block: 4
    blocks = torch.tensor([bad, [0, 2, 4]], dtype=torch.int32)
    o, lse = mods[dtype].attn_paged_sparse(c.batch(), c.q_abs, c.q_rope, blocks.cuda())
    flagged(mods[dtype], 1 << 8)
    blocks[0] = -1
    c.check_attention(o, lse, listed_rows(c, blocks))


# ---- append -------------------------------------------------------------------------------------------------
def check_append(c, m, dims, kv, q, gains=None, in_place=False):
    before = c.cache.clone()
    sums = m.new_summaries(c.num_pages)
    sums += 5
    qd = c.on(q)
    got = m.paged_append(c.batch(), kv, q_rope=qd, q_out=qd if in_place else None, summaries=sums)
    ok(m)
    assert (got is qd) == in_place
    half, W, d_c = HALF[c.dtype], c.W, dims.d_c
    x = kv.double().cpu()
    written = torch.zeros(before.shape[:2], dtype=torch.bool)
    after = c.cache.double().cpu()
    for t, b, pos in c.tokens():
        page, r = int(c.table[b, pos // c.page]), pos % c.page
        written[page, r] = True
        want = x[t].clone()
        if gains is not None:
            want[:d_c] = want[:d_c] / (want[:d_c].square().mean() + 1e-6).sqrt() * gains.double()
        want[d_c:] = rope(want[d_c:], pos, dims)
        tol = torch.zeros(W, dtype=torch.float64)
        # norm: 512 squares, a root and two products in fp32; rotation: two products and a sum of them; one rounding
        tol[:d_c] = (half + (600 * 2.0 ** -24 if gains is not None else 0)) * want[:d_c].abs() if gains is not None else 0
        pair = x[t][d_c:].view(-1, 2).norm(dim=1).repeat_interleave(2) * 1.5
        tol[d_c:] = half * want[d_c:].abs() + 8 * 2.0 ** -24 * pair
        assert ((after[page, r] - want).abs() <= tol).all(), (t, b, pos)
        tol = half * 2.0 * q[t].abs().max() + 8 * 2.0 ** -24
        wq = rope(q[t], pos, dims)
        pair = q[t].view(c.dims.n_h, -1, 2).norm(dim=-1).repeat_interleave(2, dim=-1) * 1.5
        tol = half * wq.abs() + 8 * 2.0 ** -24 * pair
        assert ((got[t].double().cpu() - wq).abs() <= tol).all(), (t, b, pos)
    same = ~written.to(c.cache.device)
    i = DT[c.dtype] == torch.bfloat16 and torch.int16 or torch.int32
    assert torch.equal(c.cache.view(i)[same], before.view(i)[same])
    if c.pad:
        assert torch.equal(got[c.T:], qd[c.T:]) if in_place else True
    # the pages that the new tokens completed, from the rows that the cache holds now; no other page
    done = sorted({int(c.table[b, pos // c.page]) for _, b, pos in c.tokens() if pos % c.page == c.page - 1})
    rest = torch.tensor([p for p in range(c.num_pages) if p not in done])
    assert (sums.cpu()[rest] == 5).all()
    if done:
        means = (after[done].sum(1) / c.page).float()
        assert torch.equal(sums.cpu()[done], c.summaries(means.double()))


@pytest.mark.parametrize("dtype,page,lens,tq,pad", [
    ("fp32", 16, [1, 16, 33, 40], [1, 16, 2, 0], 0), ("bf16", 16, [1, 16, 33, 40], [1, 16, 2, 0], 3),
    ("bf16", 64, [64, 4096, 65, 128, 100], [1, 1, 1, 1, 1], 0), ("bf16", 64, [1000, 200], [700, 137], 5),
    ("bf16", 48, [500], [333], 0), ("fp32", 32, [131072 + 32], [40], 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(mods, dtype, page, lens, tq, pad, in_place):
    c = Case(dtype, page, lens, tq, seed=20, pad=pad)
    wide = torch.full((c.T + pad, c.W + 16), 3.0, dtype=DT[dtype], device="cuda")   # rows of a wider projection
    kv = wide[:, :c.W]
    kv.copy_(c.normal(c.T + pad, c.W))
    check_append(c, mods[dtype], c.dims, kv, c.normal(c.T + pad, c.dims.n_h, c.dims.d_r), in_place=in_place)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_with_norm_and_yarn(dtype):
    c = Case(dtype, 32, [131072, 70, 5], [3, 40, 5], seed=21)
    m = handle(dtype)
    dims = synth.Dims(**{**c.dims.__dict__, "yarn_s": 40.0, "yarn_l0": 4096.0})
    mla.mla_set_yarn(m.handle, 40.0, dims.yarn_alpha, dims.yarn_beta, 4096.0)
    gq, gkv = c.on(c.normal(c.dims.d_cq)), c.normal(c.dims.d_c)
    gd = c.on(gkv)
    mla.mla_set_rmsnorm(m.handle, gq, gd, 1e-6)
    check_append(c, m, dims, c.on(c.normal(c.T, c.W)), c.normal(c.T, c.dims.n_h, c.dims.d_r), gains=gkv)
    m.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_flags_bad_pages_and_writes_nothing_for_them(mods, dtype):
    m = mods[dtype]
    c = Case(dtype, 16, [40, 20], [20, 1], seed=22)
    c.d_table[0, 1] = c.num_pages
    page2 = int(c.table[0, 2])
    before = c.cache.clone()
    kv = c.on(c.normal(c.T, c.W))
    m.paged_append(c.batch(), kv)
    flagged(m, 1 << 7)
    i = torch.int16 if dtype == "bf16" else torch.int32
    changed = (c.cache.view(i) != before.view(i)).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == sorted([page2, int(c.table[1, 1])])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,tq,pad", [([33, 20], [2, 1], 1), ([64, 5, 300], [64, 0, 7], 40), ([1], [1], 299)])
def test_append_leaves_query_rows_behind_the_last_sequence(mods, dtype, in_place, lens, tq, pad):
    m = mods[dtype]
    c = Case(dtype, 16, lens, tq, seed=25, pad=pad)
    qd = c.q_rope
    out = qd if in_place else torch.full_like(qd, 7.0)
    before = out.clone()
    m.paged_append(c.batch(), c.on(c.normal(c.T + pad, c.W)), q_rope=qd, q_out=out, summaries=m.new_summaries(c.num_pages))
    ok(m)
    assert torch.equal(out[c.T:], before[c.T:])
    last = c.tokens()[-1][0]
    assert c.tokens()[-1][2] == 0 or not torch.equal(out[last], before[last])       # (position 0 is not turned)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_summaries_of_values_far_apart(mods, dtype, page):
    """Rows whose values span 120 binades, half of them cancelled by their negatives: sums that a double rounds."""
    m = mods[dtype]
    c = Case(dtype, page, [page], [1], seed=24)
    d = c.dims
    x = c.normal(page, c.W) * 2.0 ** (torch.randint(-60, 61, (page, c.W), generator=c.g).double())
    x[page // 2:page - page // 4] = -x[:page // 4]
    x = x.to(DT[dtype])
    p = int(c.table[0, 0])
    c.cache[p] = x.cuda()
    sums = m.new_summaries(c.num_pages)
    m.paged_append(c.batch(), c.on(x[-1:].double()), summaries=sums)
    ok(m)
    rows = c.cache[p].double().cpu()                       # (the last row's rotary part has been turned)
    mean = torch.tensor([math.fsum(col) / page for col in rows.T.tolist()], dtype=torch.float64)
    # page additions in 53 bits, the division and the rounding to fp32 (half a step each)
    off = page * 2.0 ** -53 * rows.abs().sum(0) / page + (2.0 ** -53 + 2.0 ** -24) * mean.abs()
    out = sums[p].cpu()
    codes, scale = out[:c.W].view(torch.int8).double(), float(out[c.W:c.W + 4].view(torch.float32))
    big = float(mean.abs().max())
    assert abs(scale - big / 127) <= (float(off.max()) + 2.0 ** -24 * big) / 127 * (1 + 2.0 ** -20)
    # the nearest whole number of scales, the division off by half a step of a quotient of up to 127
    assert ((codes * scale - mean).abs() <= scale / 2 + off + 128 * 2.0 ** -24 * scale).all()
    assert codes.abs().max() == 127


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_gives_flagged_tokens_empty_queries(mods, dtype, in_place):
    """The middle sequence has fewer rows than new tokens, so its queries come back as zeros; the others are rotated,
    the rows behind the last sequence stay as they were, and no page is complete."""
    m = mods[dtype]
    c = Case(dtype, 16, [40, 20, 9], [3, 2, 1], seed=23, pad=4)
    c.d_lens[1] = 1
    d, q = c.dims, c.q[..., c.dims.d_c:]
    kv, qd, cache, sums = c.on(c.normal(c.T + 4, c.W)), c.q_rope, c.cache.clone(), m.new_summaries(c.num_pages) + 5
    out = qd if in_place else torch.full_like(qd, 7.0)
    kept = out[c.T:].clone()
    assert m.paged_append(c.batch(), kv, q_rope=qd, q_out=out, summaries=sums) is out
    flagged(m, 1 << 1)
    got = out.double().cpu()
    assert (got[3:5] == 0).all() and torch.equal(out[c.T:], kept) and (sums == 5).all()
    rows = [(int(c.table[b, pos // 16]), pos % 16) for t, b, pos in c.tokens() if b != 1]
    for t, b, pos in c.tokens():
        if b != 1:
            # as in check_append: one rounding of the result, two products and their sum in fp32
            want = rope(q[t], pos, d)
            pair = q[t].view(d.n_h, -1, 2).norm(dim=-1).repeat_interleave(2, dim=-1) * 1.5
            assert ((got[t] - want).abs() <= HALF[dtype] * want.abs() + 8 * 2.0 ** -24 * pair).all(), (t, b, pos)
    i = torch.int16 if dtype == "bf16" else torch.int32
    changed = (c.cache.view(i) != cache.view(i)).any(-1).nonzero().tolist()
    assert sorted(map(tuple, changed)) == sorted(rows)


# ---- selection ----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,page,lens,tq,top_k,first,last", [
    ("fp32", 16, [700, 90, 16], [3, 2, 1], 8, 1, 2), ("bf16", 16, [700, 90, 16], [3, 2, 1], 8, 1, 2),
    ("bf16", 16, [9000, 3000], [1, 1], 64, 0, 1), ("bf16", 64, [9000], [70], 16, 2, 3),
    ("bf16", 16, [2100, 2000], [130, 5], 1, 0, 1), ("bf16", 32, [5000], [2], 7, 3, 4),
    ("bf16", 16, [16 * 300], [1], 200, 1, 1)])
def test_select(mods, dtype, page, lens, tq, top_k, first, last):
    m = mods[dtype]
    c = Case(dtype, page, lens, tq, seed=top_k + page, pad=2)
    means = c.normal(c.num_pages, c.W) * 0.3
    blocks = torch.full((c.T + 2, top_k), -9, dtype=torch.int32, device="cuda")
    m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), top_k, first, last, blocks)
    ok(m)
    assert torch.equal(blocks[:c.T].cpu(), c.select(means, top_k, first, last))
    assert (blocks[c.T:] == -9).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_select_ties_and_empty_summaries(mods, dtype):
    m = mods[dtype]
    c = Case(dtype, 16, [16 * 150, 16 * 40], [2, 1], seed=30)
    means = c.normal(3, c.W)[torch.arange(c.num_pages) % 3]             # three kinds of pages: ties everywhere
    means[c.table[0, 7].long()] = 0
    means[c.table[0, 9].long(), 3] = float("inf")                       # scale 0, codes 0
    for top_k, first, last in ((20, 1, 1), (100, 0, 2), (3, 0, 1)):
        got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), top_k, first, last)
        ok(m)
        assert torch.equal(got.cpu(), c.select(means, top_k, first, last))
    c.q[:] = 0                                                          # nothing to tell them apart
    got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), 20, 1, 2)
    ok(m)
    assert torch.equal(got.cpu(), c.select(means, 20, 1, 2))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_select_queries_out_of_range(mods, dtype):
    """Heads of zeros, of tiny and huge values, with an infinity and with a NaN: scale 0 where none is finite."""
    m = mods[dtype]
    c = Case(dtype, 16, [16 * 200], [1], seed=31)
    means = c.normal(c.num_pages, c.W) * 0.3
    d = c.dims
    c.q *= 1e-3
    c.q[0, 0] *= 1e33
    c.q[0, 1] = float("inf")
    c.q[0, 2, 5] = float("nan")
    c.q[0, 3] = 0
    c.q[0, 0, 7] = -float("inf") if d.n_h > 100 else c.q[0, 0, 7]
    c.q = c.q.to(DT[dtype]).double()
    for tiny in (1.0, 1e-37):
        c.q = (c.q * tiny).to(DT[dtype]).double()
        got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), 20, 1, 2)
        ok(m)
        assert torch.equal(got.cpu(), c.select(means, 20, 1, 2)), tiny


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_select_half_of_the_largest(mods, dtype):
    """Elements at every half step of the scale: the ties of the rounding, one way or the other by the scale's own."""
    m = mods[dtype]
    c = Case(dtype, 16, [16 * 300], [2], seed=32)
    top = torch.rand(2, c.dims.n_h, 1, generator=c.g, dtype=torch.float64) + 0.5
    c.q = (top * (torch.randint(-127, 128, c.q.shape, generator=c.g) + 0.5) / 127).to(DT[dtype]).double()
    c.q[..., 0] = top[..., 0].to(DT[dtype]).double()
    c.q[..., 1] = -c.q[..., 0] / 2
    c.q[..., -1] = c.q[..., 0] / 2
    means = c.normal(c.num_pages, c.W)
    got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), 33, 0, 1)
    ok(m)
    assert torch.equal(got.cpu(), c.select(means, 33, 0, 1))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_select_over_many_sequences(mods, dtype):
    """More sequences than one look at cu_q takes, empty ones and a flagged one among them; some see fewer blocks
    than top_k."""
    m = mods[dtype]
    tq = [(3 * b) % 5 % 4 for b in range(300)]
    c = Case(dtype, 16, [20 + (37 * b) % 150 for b in range(300)], tq, seed=33)
    bad = 204
    assert tq[bad] == 2
    c.d_lens[bad] = 1                                                   # fewer rows than new tokens
    means = c.normal(c.num_pages, c.W)
    got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), 5, 1, 2)
    flagged(m, 1 << 1)
    want = c.select(means, 5, 1, 2)
    want[int(c.cu[bad]):int(c.cu[bad + 1])] = -1
    assert torch.equal(got.cpu(), want)


def test_select_runs_that_cross_sequences(mods):
    """Several tokens and both tiles of 128 blocks in one CTA, with the ends of sequences between them."""
    c = Case("bf16", 16, [3300, 40, 2500, 2200, 2060], [150, 1, 120, 0, 81], seed=34)
    means = c.normal(c.num_pages, c.W) * 0.3
    got = mods["bf16"].paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), 9, 1, 2)
    ok(mods["bf16"])
    assert torch.equal(got.cpu(), c.select(means, 9, 1, 2))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("top_k", [50, 8300])
def test_select_among_more_blocks_than_shared_memory_holds(mods, dtype, top_k):
    """8391 blocks over 41 pages, so that scores tie in hundreds."""
    m = mods[dtype]
    c = Case(dtype, 16, [16 * 41], [2], seed=35, spare=0)
    nb = 8391
    c.table = c.table[:, torch.arange(nb) * 7 % 41].contiguous()
    c.lens = [16 * nb]
    c.d_table, c.d_lens = c.table.cuda(), torch.tensor(c.lens, device="cuda")
    means = c.normal(c.num_pages, c.W)
    got = m.paged_select(c.batch(), c.q_abs, c.q_rope, c.summaries(means).cuda(), top_k, 1, 2)
    ok(m)
    assert torch.equal(got.cpu(), c.select(means, top_k, 1, 2))


# ---- together -----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_prompt_in_chunks_then_decode_steps(mods, dtype):
    """Chunks of a prompt, then single tokens: append, choose blocks, attend, with the cache and the summaries
    carried along; every step against the float64 form over the rows that the cache holds."""
    m = mods[dtype]
    page, top_k = 16, 6
    c = Case(dtype, page, [150, 90], [150, 90], seed=40)
    d = c.dims
    c.cache.fill_(NAN)
    sums = m.new_summaries(c.num_pages)
    full = [c.normal(n, c.W) for n in c.lens]
    at = [0, 0]
    for new in ([100, 17], [30, 60], [1, 1], [1, 0], [1, 1], [17, 11]):
        new = [min(n, len(full[b]) - at[b]) for b, n in enumerate(new)]
        at = [a + n for a, n in zip(at, new)]
        c.lens, c.tq, c.T = list(at), list(new), sum(new)
        c.cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
        c.d_cu, c.d_lens = c.cu.cuda(), torch.tensor(at, dtype=torch.int64, device="cuda")
        c.q = c.normal(c.T, d.n_h, c.W)
        kv = c.on(torch.cat([full[b][at[b] - n:at[b]] for b, n in enumerate(new)]))
        q_rope = m.paged_append(c.batch(), kv, q_rope=c.q_rope, summaries=sums)
        c.q[..., d.d_c:] = q_rope.double().cpu()
        qa = c.q_abs
        blocks = m.paged_select(c.batch(), qa, q_rope, sums, top_k, 1, 2)
        o, lse = m.attn_paged_sparse(c.batch(), qa, q_rope, blocks)
        o2, lse2 = m.attn_paged(c.batch(), qa, q_rope)
        ok(m)
        pool = c.cache.double().cpu()
        c.rows = []
        for b, n in enumerate(at):
            pos = torch.arange(n)
            c.rows.append(pool[c.table[b, pos // page].long(), pos % page])
        means = (pool.sum(1) / page).float().double()                    # of whole pages; the others are forced
        assert torch.equal(blocks.cpu(), c.select(torch.nan_to_num(means), top_k, 1, 2))
        c.check_attention(o, lse, listed_rows(c, blocks.cpu()))
        c.check_attention(o2, lse2, prefix(c))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_captured_steps_replay_on_new_lengths(mods, dtype):
    """Two graphs of the same handle, captured one after the other and replayed in turn with other lengths,
    tables and a batch that shrank (its last rows padded)."""
    m = mods[dtype]
    a, b = (Case(dtype, 32, [300, 64], [2, 2], seed=50 + k) for k in range(2))
    state = []
    for c in (a, b):
        kv, qa, qr = c.on(c.normal(c.T, c.W)), c.q_abs, c.q_rope
        sums, blocks = c.summaries(c.normal(c.num_pages, c.W)).cuda(), torch.empty(c.T, 4, dtype=torch.int32, device="cuda")
        o, lse = torch.empty_like(qa), torch.empty(c.T, c.dims.n_h, device="cuda")
        batch = c.batch()

        def step(c=c, kv=kv, qa=qa, qr=qr, sums=sums, blocks=blocks, o=o, lse=lse, batch=batch):
            m.paged_append(batch, kv, summaries=sums)
            m.paged_select(batch, qa, qr, sums, 4, 1, 1, blocks)
            m.attn_paged_sparse(batch, qa, qr, blocks, o, lse)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        state.append((c, g, kv, qa, qr, sums, blocks, o, lse))
    m.workspace(1 << 26)                                    # a larger call in between
    for lens, tq in (([299, 64], [2, 2]), ([200, 33], [1, 2]), ([97, 50], [3, 0])):
        for c, g, kv, qa, qr, sums, blocks, o, lse in state:
            c.lens, c.tq, c.T = list(lens), list(tq), sum(tq)
            c.cu = torch.tensor([0] + tq, dtype=torch.int64).cumsum(0)
            c.d_cu.copy_(c.cu)
            c.d_lens.copy_(torch.tensor(lens))
            o.fill_(7.0)
        for _, g, *_ in state:
            g.replay()
        torch.cuda.synchronize()
        ok(m)
        for c, g, kv, qa, qr, sums, blocks, o, lse in state:
            pool = c.cache.double().cpu()
            c.rows = [pool[c.table[s, torch.arange(n) // 32].long(), torch.arange(n) % 32] for s, n in enumerate(lens)]
            c.check_attention(o, lse, listed_rows(c, blocks.cpu()))
            assert (o[c.T:] == 7).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 100])
def test_a_batch_without_new_tokens_leaves_everything_as_it_was(mods, dtype, T):
    m = mods[dtype]
    c = Case(dtype, 16, [100, 0, 33], [0, 0, 0], seed=61, pad=T)
    d = c.dims
    cache, kv = c.cache.clone(), c.on(c.normal(T, c.W))
    sums = m.new_summaries(c.num_pages) + 5
    q_out = torch.full((T, d.n_h, d.d_r), 7.0, dtype=DT[dtype], device="cuda")
    blocks = torch.full((T, 4), -9, dtype=torch.int32, device="cuda")
    o = torch.full((T, d.n_h, d.d_c), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, d.n_h), 7.0, device="cuda")
    m.paged_append(c.batch(), kv, q_rope=c.q_rope, q_out=q_out, summaries=sums)
    m.paged_select(c.batch(), c.q_abs, c.q_rope, sums, 4, 1, 1, blocks)
    m.attn_paged(c.batch(), c.q_abs, c.q_rope, o, lse)
    m.attn_paged_sparse(c.batch(), c.q_abs, c.q_rope, blocks, o, lse)
    ok(m)
    i = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(c.cache.view(i), cache.view(i)) and (sums == 5).all()
    assert all((x == y).all() for x, y in ((q_out, 7), (blocks, -9), (o, 7), (lse, 7)))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_pages_far_into_a_large_pool(mods, dtype):
    """Rows whose element offsets pass 2^32: every call at the end of a pool of 9 GB."""
    m = mods[dtype]
    c = Case(dtype, 64, [300, 64, 190], [3, 1, 62], seed=64)
    d, far = c.dims, 9 * 2 ** 30 // (64 * c.W * c.cache.element_size())
    assert far * 64 * c.W > 2 ** 31
    small, c.cache = c.cache, torch.empty(far + c.num_pages, 64, c.W, dtype=DT[dtype], device="cuda")
    c.cache[far:] = small
    c.d_table = c.d_table + far * (c.d_table >= 0).int()
    kv, sums = c.on(c.normal(c.T, c.W)), m.new_summaries(far + c.num_pages)
    q_rope = m.paged_append(c.batch(), kv, q_rope=c.q_rope, summaries=sums)
    c.q[..., d.d_c:] = q_rope.double().cpu()
    blocks = m.paged_select(c.batch(), c.q_abs, q_rope, sums, 3, 0, 1)
    o, lse = m.attn_paged(c.batch(), c.q_abs, q_rope)
    o2, lse2 = m.attn_paged_sparse(c.batch(), c.q_abs, q_rope, blocks)
    ok(m)
    pool = c.cache[far:].double().cpu()
    c.rows = [pool[c.table[b, torch.arange(n) // 64].long(), torch.arange(n) % 64] for b, n in enumerate(c.lens)]
    c.check_attention(o, lse, prefix(c))
    c.check_attention(o2, lse2, listed_rows(c, blocks.cpu()))
    done = sorted({int(c.table[b, pos // 64]) for _, b, pos in c.tokens() if pos % 64 == 63})
    assert torch.equal(sums[far:].cpu()[done], c.summaries((pool[done].sum(1) / 64).float().double()))
    assert not sums[:far].any()


@pytest.mark.parametrize("dtype,times", [("fp32", 16), ("bf16", 1024)])
def test_attention_over_a_long_table_of_the_same_pages(mods, dtype, times):
    """The same 1024 rows over and over: the same weighted mean, ln(times) more in the logarithm of the sum."""
    m = mods[dtype]
    c = Case(dtype, 64, [1024], [1], seed=65, spare=0)
    n = 1024 * times
    b = mla.PagedBatch(c.cache, c.d_table[:, :16].repeat(1, times), c.d_cu, torch.tensor([n], device="cuda"), 1)
    o, lse = m.attn_paged(b, c.q_abs, c.q_rope)
    ok(m)
    ro, rl, A, gamma = c.attend(0, c.rows[0])
    # as in check_attention; bf16 sums 4096 steps of 256 rows in 74 ranges, then the 74 partials
    terms = n if dtype == "fp32" else 56 * 256 + 74
    rel = 2 * gamma + 2.0 ** -18 + terms * 2.0 ** -23 + (HALF["bf16"] if dtype == "bf16" else 0.0)
    assert ((o[0].double().cpu() - ro).abs() <= rel[:, None] * A + HALF[dtype] * ro.abs() * (1 + rel[:, None])).all()
    want = rl + torch.tensor(float(times), dtype=torch.float64).log()
    assert ((lse[0].double().cpu() - want).abs() <= gamma + 2.0 ** -18 + terms * 2.0 ** -23 + 2.0 ** -23 * want.abs()).all()


def test_attention_over_pieces_that_take_seconds(mods):
    """A token a pair, each over 3 * 2^26 rows, 1024 rows over and over: 786432 steps, of 4357 cycles at least (the MMAs'),
    are 3.4e9 cycles, more than one wait may take. Nothing gives up, and the sums are those of all rows."""
    m = mods["bf16"]
    T, times = torch.cuda.get_device_properties(0).multi_processor_count // 2, 3 * 2 ** 16
    c = Case("bf16", 64, [1024], [1], seed=70, spare=0, pad=T - 1)
    n = 1024 * times
    b = mla.PagedBatch(c.cache, c.d_table[:, :16].repeat(1, times), torch.tensor([0, T], device="cuda"),
                       torch.tensor([n], device="cuda"), T)
    o, lse = m.attn_paged(b, c.q_abs, c.q_rope)
    ok(m)
    assert torch.isfinite(o).all()
    for t in (0, 1, T - 2, T - 1):
        _, rl, _, gamma = c.attend(t, c.rows[0])
        # the T - 1 - t rows that t does not see are part of one of the `times` rounds. A thread adds 786432 sums of 64
        # weights, to partial sums that grow evenly to the whole; 2^-18 for the exponentials
        rel = (n / 256 / 2 + 64) * 2.0 ** -23 + 2.0 ** -18 + 2.0 / times
        want = rl + torch.tensor(float(times), dtype=torch.float64).log()
        err = (lse[t].double().cpu() - want).abs()
        assert (err <= gamma + rel + 2.0 ** -23 * want.abs()).all(), (t, float(err.max()))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_calls_and_graphs_side_by_side_on_two_streams(mods, dtype):
    """The same calls of one handle on two streams at once, eager and as two graphs: as when they run alone."""
    m = mods[dtype]
    cases = [Case(dtype, 16, lens, tq, seed=60 + k) for k, (lens, tq) in enumerate((([900, 64, 33], [3, 1, 2]),
                                                                                 ([16 * 200], [40])))]
    jobs = []
    for c in cases:
        qa, qr, sums = c.q_abs, c.q_rope, c.summaries(c.normal(c.num_pages, c.W)).cuda()
        blocks = torch.empty(c.T, 6, dtype=torch.int32, device="cuda")
        outs = [torch.empty_like(qa), torch.empty(c.T, c.dims.n_h, device="cuda"),
                torch.empty_like(qa), torch.empty(c.T, c.dims.n_h, device="cuda")]

        def step(batch=c.batch(), qa=qa, qr=qr, sums=sums, blocks=blocks, outs=outs):
            m.paged_select(batch, qa, qr, sums, 6, 1, 1, blocks)
            m.attn_paged_sparse(batch, qa, qr, blocks, *outs[:2])
            m.attn_paged(batch, qa, qr, *outs[2:])
        step()
        ok(m)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        torch.cuda.synchronize()
        jobs.append((step, g, torch.cuda.Stream(), [blocks, *outs], [x.clone() for x in (blocks, *outs)]))
    for graphs in (False, True):
        for _, _, _, got, _ in jobs:
            for x in got:
                x.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for step, g, s, _, _ in jobs:
                with torch.cuda.stream(s):
                    g.replay() if graphs else step()
        torch.cuda.synchronize()
        ok(m)
        for _, _, _, got, want in jobs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))
