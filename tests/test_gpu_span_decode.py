"""smla_decode_spans through the binding against 64-bit attention (needs a B200): whole sequences and
listed spans, ragged batches, empty requests, bad pages, streams, graphs and waits that run out.
The caches are NaN bytes wherever no request has a token."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_fp8_b200 as smla
from sparse_mla_decode_fp8_b200 import build
from tests import independent
from tests import span_util as U
from sparse_mla_decode_fp8_b200 import workloads as W

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    build.build()
    smla.library()


def _queries(B, seed):
    return W.to_bf16_bits(np.random.default_rng(seed).standard_normal((B, 64, 512)).astype(np.float32))


def _workspace(B):
    # everything but the error word may hold anything
    ws = torch.full((smla.decode_spans_workspace_bytes(B),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    return ws


def _run(lens, seed, spans=None, sm_scale=SCALE, **kw):
    cache, table = U.paged(lens, seed)
    qb = _queries(len(lens), seed)
    ws = _workspace(len(lens))
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.asarray(lens, np.int32)), sm_scale,
                                 spans=None if spans is None else U.dev(np.asarray(spans, np.int32)), workspace=ws, **kw)
    torch.cuda.synchronize()
    assert smla.read_error(ws) == 0
    positions = []
    for b, n in enumerate(lens):
        if spans is None:
            positions.append(np.arange(max(n, 0)))
        else:
            p = (np.asarray(spans[b], np.int64)[:, None] * 64 + np.arange(64)).reshape(-1)
            positions.append(p[(p >= 0) & (p < n)])
    U.check_decode(out, lse, independent.q_values(qb), cache, table, positions, sm_scale)
    return out, lse


@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000])
def test_one_request(length):
    _run([length], seed=length)


def test_one_long_request_over_every_sm():
    _run([40000], seed=1)


@pytest.mark.parametrize("lens", [[0], [0, 0, 5, 0], [-7, 300], [130, 0, 1, 64, 129, 0, 0, 2000, 31],
                                  [1500, 1, 1, 700, 3000, 128, 256, 384]])
def test_ragged(lens):
    _run(lens, seed=len(lens) + lens[-1])


def test_more_requests_than_sms():
    rng = np.random.default_rng(3)
    _run(list(rng.integers(0, 400, 333)), seed=3)


def test_requests_of_several_tiles_inside_one_cta():
    # 700 requests of 1..2 tiles: each CTA walks several whole ones
    rng = np.random.default_rng(4)
    _run(list(rng.integers(1, 200, 700)), seed=4)


@pytest.mark.parametrize("sm_scale", [0.0, -SCALE, 8.0])
def test_scales(sm_scale):
    # 8: one token takes nearly all the weight, and the reference moves often
    _run([777, 130], seed=5, sm_scale=sm_scale)


def test_rising_scores_move_the_reference():
    # later tokens point ever more along the query: every tile raises the maxima
    n = 1300
    cache, table = U.paged([n], seed=6)
    qb = _queries(1, 6)
    q = independent.q_values(qb)
    mean = np.sign(q[0, 0]).astype(np.float32)
    W.write_tokens(cache, table[0, np.arange(n) // 256].astype(np.int64), np.arange(n) % 256,
                   (np.arange(n, dtype=np.float32)[:, None] / 20) * mean)
    ws = _workspace(1)
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array([n], np.int32)), 0.05, workspace=ws)
    U.check_decode(out, lse, q, cache, table, [np.arange(n)], 0.05)


@pytest.mark.parametrize("nsel", [1, 2, 3, 7, 32, 129])
def test_listed_spans(nsel):
    lens = [5000, 100, 0, 1, 4096, 20000]
    rng = np.random.default_rng(nsel)
    spans = np.full((len(lens), nsel), -1, np.int32)
    for b, n in enumerate(lens):
        have = -(-n // 64)
        k = min(nsel, have)
        spans[b, :k] = rng.choice(max(have, 1), k, replace=False)
        rng.shuffle(spans[b])
    _run(lens, seed=nsel, spans=spans)


def test_listed_spans_repeat_and_out_of_range():
    spans = [[3, 3, 0, -1, 3], [4, 5, 1 << 24, -5, 2**31 - 1], [-1, -1, -1, -1, -1], [0, 0, 0, 0, 0]]
    _run([250, 257, 600, 0], seed=8, spans=spans)


def test_a_sequence_longer_than_its_table_is_cut():
    cache, table = U.paged([512], seed=9)
    qb = _queries(1, 9)
    ws = _workspace(1)
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array([2**31 - 1], np.int32)), SCALE,
                                 workspace=ws)
    assert smla.read_error(ws) == 0
    U.check_decode(out, lse, independent.q_values(qb), cache, table, [np.arange(512)], SCALE)


def test_bad_pages_hold_no_tokens_and_are_reported():
    lens = [700, 300, 256]
    cache, table = U.paged(lens, seed=10)
    table[0, 1], table[2, 0] = len(cache), -1
    qb = _queries(3, 10)
    ws = _workspace(3)
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE, workspace=ws)
    assert smla.read_error(ws) == smla.SMLA_FLAG_BAD_PAGE
    U.check_decode(out, lse, independent.q_values(qb), cache, table,
                   [np.r_[0:256, 512:700], np.arange(300), np.arange(0)], SCALE)


def test_equals_the_sparse_decode_over_the_same_tokens():
    lens, nsel = [3000, 900], 8
    cache, table = U.paged(lens, seed=11)
    qb = _queries(2, 11)
    d = [U.dev(cache), U.dev(table)]
    x = torch.rand((2, 48), device="cuda")
    sl = U.dev(np.array(lens, np.int32))
    spans, idx = smla.select_spans(x, sl, nsel, keep_first=1, keep_last=1)
    out, lse = smla.decode_spans(U.dev_bf16(qb), *d, sl, SCALE, spans=spans)
    ref, ref_lse = smla.decode(U.dev_bf16(qb), *d, idx, sl, SCALE)
    assert (lse - ref_lse).abs().max() <= 1e-5 * (1 + ref_lse.abs().max())
    # one side rounds its weights and its output to bf16, 2^-9 of each in the mean, the other to two bf16
    # terms and fp32: 2^-9 sqrt(2) = 2.8e-3 of the norm, below 5e-3
    assert (out.double() - ref.double()).norm() <= 5e-3 * ref.double().norm()


def test_results_repeat_bit_for_bit_and_leave_other_rows():
    lens = np.array([3001, 77, 0, 513], np.int32)
    cache, table = U.paged(lens, seed=12)
    qb = _queries(4, 12)
    args = (U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(lens), SCALE)
    out = torch.full((6, 64, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 64), 9.0, device="cuda")
    first = [t.clone() for t in smla.decode_spans(*args, out=out[:4], lse=lse[:4], workspace=_workspace(4))]
    assert (out[4:] == 9.0).all() and (lse[4:] == 9.0).all()
    for _ in range(3):
        again = smla.decode_spans(*args)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_another_stream_and_a_replayed_graph_with_new_lengths():
    lens = np.array([900, 2000], np.int32)
    cache, table = U.paged([2000, 2000], seed=13)
    qb = _queries(2, 13)
    q, c, t, sl = U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = smla.decode_spans(q, c, t, sl, SCALE, stream=side)
    side.synchronize()
    qv = independent.q_values(qb)
    U.check_decode(out, lse, qv, cache, table, [np.arange(n) for n in lens], SCALE)
    ws = _workspace(2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = smla.decode_spans(q, c, t, sl, SCALE, workspace=ws)
    for lens in ([2000, 1], [0, 130], [5, 1999]):
        sl.copy_(U.dev(np.array(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        U.check_decode(out, lse, qv, cache, table, [np.arange(n) for n in lens], SCALE)


@pytest.mark.parametrize("lens", [[100], [1000, 50], [40000, 1, 300]])
def test_a_wait_that_runs_out_is_reported_and_leaves_nan_rows(lens):
    # the first score MMAs signal a barrier nobody waits for: every CTA with tiles runs out of its 2 ms
    cache, table = U.paged(lens, seed=14)
    qb = _queries(len(lens), 14)
    args = (U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    ws = _workspace(len(lens))
    out, lse = smla.decode_spans(*args, workspace=ws, wait_timeout_ns=2_000_000, debug_flags=smla.SMLA_DEBUG_SKIP_FIRST_COMMIT)
    torch.cuda.synchronize()
    assert smla.read_error(ws) & smla.SMLA_FLAG_TIMEOUT
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = smla.decode_spans(*args, workspace=ws)
    assert smla.read_error(ws) == 0
    U.check_decode(out, lse, independent.q_values(qb), cache, table, [np.arange(n) for n in lens], SCALE)


def test_refusals():
    cache, table = U.paged([300], seed=15)
    q, c, t = U.dev_bf16(_queries(1, 15)), U.dev(cache), U.dev(table)
    sl = U.dev(np.array([300], np.int32))
    for bad in (dict(spans=torch.zeros((2, 3), dtype=torch.int32, device="cuda")), dict(spans=torch.zeros((1, 0), dtype=torch.int32, device="cuda")),
                dict(spans=torch.zeros((1, 1025), dtype=torch.int32, device="cuda")), dict(out=torch.empty((1, 64, 512), device="cuda")),
                dict(lse=torch.empty((1, 63), device="cuda")), dict(workspace=torch.zeros(1000, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(smla.SmlaError):
            smla.decode_spans(q, c, t, sl, SCALE, **bad)
    for args in ((q.float(), c, t, sl), (q[:, :32], c, t, sl), (q, c[:, :-16], t, sl), (q, c, t.long(), sl), (q, c, t, sl.cpu())):
        with pytest.raises(smla.SmlaError):
            smla.decode_spans(*args, SCALE)
    with pytest.raises(smla.SmlaError):
        smla.decode_spans(q, c, t, sl, float("nan"))


def test_single_tokens_come_back_exactly_for_every_code_and_scale_byte():
    # 255 requests of one token each, q = 0: the weight is 1 and the result the token itself.  Group g of request s
    # has scale byte (s + 37 g) mod 255, dims cycle through the e4m3 codes; at scale bytes above 246 through
    # those below 2, so that every value lies in the bf16 range.
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    small = np.array([c for c in range(256) if c & 0x7F < 0x40], np.uint8)
    cache = np.full((255, W.PAGE_BYTES), 0xFF, np.uint8)
    rows, scales = W.row_views(cache)
    rng = np.random.default_rng(1)
    s = (np.arange(255)[:, None] + 37 * np.arange(7)) % 255
    scales[:, 0, :7] = s
    for g in range(7):
        at = 64 * g + np.arange(64) + 13 * np.arange(255)[:, None]
        rows[:, 0, 64 * g:64 * g + 64] = np.where(s[:, g:g + 1] > 246, small[at % len(small)], codes[at % len(codes)])
    rows[:, 0, 448:] = W.to_bf16_bits(rng.standard_normal((255, 64)).astype(np.float32)).view(np.uint8).reshape(255, 128)
    table = np.arange(255, dtype=np.int32)[:, None]
    ws = _workspace(255)
    out, lse = smla.decode_spans(torch.zeros((255, 64, 512), dtype=torch.bfloat16, device="cuda"), U.dev(cache), U.dev(table),
                                 U.dev(np.ones(255, np.int32)), SCALE, workspace=ws)
    assert smla.read_error(ws) == 0
    want = independent.token_latents(cache, np.arange(255), np.zeros(255, np.int64))
    got = out.double().cpu().numpy()
    assert (lse == 0).all() and np.array_equal(got[:, :1].repeat(64, 1), got)
    exact = np.concatenate([np.repeat(s >= 10, 64, 1), np.ones((255, 64), bool)], 1)
    assert np.array_equal(got[:, 0][exact], want[exact])
    # below scale byte 10 only what lies under the least normal number may round, by less than that number
    assert (np.abs(got[:, 0] - want) < 2.0 ** -126).all()


def test_nan_scale_nan_query_and_their_neighbours():
    # a 0xFF scale byte of one token makes its request NaN, a NaN in one head's query that head; nothing else changes
    lens = [300, 200, 1000]
    cache, table = U.paged(lens, seed=16)
    qb = _queries(3, 16)
    ref, ref_lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    W.row_views(cache)[1][table[0, 1], 5, 3] = 0xFF
    qb[1, 7, 100] = 0x7FC0
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isnan(out[1, 7]).all() and torch.isnan(lse[1, 7])
    keep = torch.arange(64, device="cuda") != 7
    assert torch.equal(out[1, keep], ref[1, keep]) and torch.equal(lse[1, keep], ref_lse[1, keep])
    assert torch.equal(out[2], ref[2]) and torch.equal(lse[2], ref_lse[2])


def test_two_calls_at_once_with_a_workspace_each():
    lens = [[3000, 500, 41], [20000]]
    calls = []
    for i, n in enumerate(lens):
        cache, table = U.paged(n, seed=17 + i)
        qb = _queries(len(n), 17 + i)
        calls.append((U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array(n, np.int32)), SCALE))
    want = [smla.decode_spans(*c) for c in calls]
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream(), torch.cuda.Stream()], [_workspace(len(n)) for n in lens]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, st, ws in zip(calls, streams, spaces):
            got.append(smla.decode_spans(*c, workspace=ws, stream=st))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    assert smla.read_error(spaces[0]) == 0 and smla.read_error(spaces[1]) == 0


def test_tensors_out_of_alignment_or_with_gaps_are_refused():
    cache, table = U.paged([300], seed=19)
    q, c, t = U.dev_bf16(_queries(1, 19)), U.dev(cache), U.dev(table)
    sl = U.dev(np.array([300], np.int32))
    shifted = torch.empty(64 * 512 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(1, 64, 512)  # 8 bytes on
    off16 = torch.zeros(c.numel() + 16, dtype=torch.uint8, device="cuda")[16:].view(c.shape)       # 32 bytes needed
    gaps = torch.zeros((1, 64, 1024), dtype=torch.bfloat16, device="cuda")[:, :, ::2]
    ws = torch.zeros(smla.decode_spans_workspace_bytes(1) + 16, dtype=torch.uint8, device="cuda")[16:]
    for args, kw in (((shifted, c, t, sl), {}), ((q, off16, t, sl), {}), ((gaps, c, t, sl), {}), ((q, c, t, sl), dict(out=shifted)),
                     ((q, c, t, sl), dict(workspace=ws)), ((q, c, t, sl), dict(out=gaps))):
        with pytest.raises(smla.SmlaError):
            smla.decode_spans(*args, SCALE, **kw)


def test_tokens_whose_scores_are_minus_infinity_weigh_nothing():
    # the last token, alone in its tile (a part of its own), has -inf in one dim where the query is positive: its
    # scores are -inf, its weight 0, and 0 times -inf makes that one dim of the output NaN, as the formula does
    n = 257
    cache, table = U.paged([n], seed=23)
    rows, scales = W.row_views(cache)
    rows[table[0, 1], 0, 64:128] = np.where(np.arange(64) == 6, 0xFE, 0)  # -448, zeros around it
    scales[table[0, 1], 0, 1] = 254  # times 2^127
    qb = _queries(1, 23)
    qb[0, :, 64:128] = 0
    qb[0, :, 70] = W.to_bf16_bits(np.ones(1, np.float32))
    d = (U.dev_bf16(qb), U.dev(cache), U.dev(table))
    out, lse = smla.decode_spans(*d, U.dev(np.array([n], np.int32)), SCALE)
    want, want_lse = smla.decode_spans(*d, U.dev(np.array([n - 1], np.int32)), SCALE)
    dims = torch.arange(512, device="cuda") != 70
    assert torch.isnan(out[0][:, ~dims]).all()
    # the same two tiles' parts, joined with one of weight 0
    assert torch.equal(out[0][:, dims], want[0][:, dims]) and torch.equal(lse, want_lse)


def test_a_request_whose_scores_are_all_minus_infinity_is_empty():
    # every token's score is -inf: ln sum exp = -inf, and no weight is left
    n = 200
    cache, table = U.paged([n], seed=24)
    rows, scales = W.row_views(cache)
    rows[table[0, 0], :n, 64:128] = np.where(np.arange(64) == 6, 0xFE, 0)
    scales[table[0, 0], :n, 1] = 254
    qb = _queries(1, 24)
    qb[0, :, 64:128] = 0
    qb[0, :, 70] = W.to_bf16_bits(np.ones(1, np.float32))
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(table), U.dev(np.array([n], np.int32)), SCALE)
    dims = torch.arange(512, device="cuda") != 70
    assert torch.isneginf(lse).all() and not out[0][:, dims].any()


@pytest.mark.parametrize("hook", [0, smla.SMLA_DEBUG_SKIP_FIRST_COMMIT])
@pytest.mark.parametrize("lens", [[100], [1000, 50, 0], [40000, 1, 300], [3000] * 200])
def test_a_limit_of_a_nanosecond(lens, hook):
    # shorter than any copy: a request is right or NaN, and the CTAs that gave up have waited for their copies and MMAs
    cache, table = U.paged(lens, seed=27)
    args = (U.dev_bf16(_queries(len(lens), 27)), U.dev(cache), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    want = smla.decode_spans(*args)
    for i in range(5):
        ws = _workspace(len(lens))
        got = smla.decode_spans(*args, workspace=ws, wait_timeout_ns=1, debug_flags=hook)
        torch.cuda.synchronize()
        flags = smla.read_error(ws)
        assert flags in (0, smla.SMLA_FLAG_TIMEOUT) and (flags or not hook)
        for b, n in enumerate(lens):
            nan = bool(torch.isnan(got[1][b]).any())
            assert nan <= (flags != 0) and (nan or not hook or n <= 0)
            for x, y in zip(got, want):
                assert torch.isnan(x[b]).all() if nan else torch.equal(x[b], y[b])
    again = smla.decode_spans(*args)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


# ---------------------------------------------------------------- many tiles in a CTA
def _tiles_per_cta(tiles):
    return -(-tiles // torch.cuda.get_device_properties(0).multi_processor_count)


def test_a_segment_moves_its_reference_three_times():
    # 300 requests share one sequence of four tiles whose scores lie 70 log2 units above each other, so that each
    # tile of a segment raises the reference and rescales what was summed.  Dims group g is nonzero in tile g only, and so
    # large there that its share, 2^-70 a raise, stays a normal number: every factor shows in the output's own digits.
    B, n = 300, 512
    assert _tiles_per_cta(B * 4) >= 8  # whole requests inside a CTA
    rng = np.random.default_rng(20)
    cache = np.full((2, W.PAGE_BYTES), 0xFF, np.uint8)
    lat = np.zeros((n, 512), np.float32)
    tile = np.arange(n) // 128
    for g in range(4):
        lat[tile == g, 64 * g:64 * g + 64] = rng.standard_normal((128, 64)) * 2.0 ** (100 - 70 * g)
    # scores: 8 rope dims that add up to the tile's height and up to two more
    lat[:, 448:456] = (70 * tile + rng.random(n) * 2).astype(np.float32)[:, None] / 8
    W.write_tokens(cache, np.arange(n) // 256, np.arange(n) % 256, lat)
    table = np.tile(np.array([[1, 0]], np.int32), (B, 1))
    cache = cache[::-1].copy()  # page 1 holds the first half
    qv = np.zeros((B, 64, 512), np.float32)
    qv[:, :, 448:456] = 1.0
    qv[:, 1::2, 448:456] = -1.0  # falling scores: the reference of the odd heads stays
    scale = float(np.log(2.0))
    ws = _workspace(B)
    out, lse = smla.decode_spans(U.dev_bf16(W.to_bf16_bits(qv)), U.dev(cache), U.dev(table), U.dev(np.full(B, n, np.int32)), scale,
                                 workspace=ws)
    assert smla.read_error(ws) == 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    o, l, mean_abs, size = U.attention(qv[0].astype(np.float64), cache, table, 0, np.arange(n), scale)
    # 8 exact products are added (the zeros add nothing), then one product and one sum in fp32, and the references'
    # roundings, each 2^-23 of the largest score at most; exp2 of both 2^-21
    e = 16 * 2.0 ** -23 * size + 2.0 ** -20
    # a request cut between two CTAs: its parts are joined by fp32 weights 2^(lambda_i - max), so that tokens whose weight
    # relative to the largest lies below the least normal number, 2^-126, may count for nothing
    k = U.latents(cache, table, 0, np.arange(n))
    s = scale * (qv[0].astype(np.float64) @ k.T)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    lost = np.minimum(p, 2.0 ** -126) @ np.abs(k)
    per = _tiles_per_cta(B * 4)
    for b in range(B):
        off = np.abs(out[b] - o)
        # an odd head's groups behind the first fall below the normal numbers: 2^-120 covers those
        bound = mean_abs * (2.0 ** -8 * (1 + 2 * e) + 2 * e + (n + 16) * 2.0 ** -23) + 2.0 ** -8 * (np.abs(o) + off) + 2.0 ** -120
        if 4 * b // per != (4 * b + 3) // per:
            bound = bound + lost
        assert (off <= bound).all(), (b, float((off / bound).max()))
        assert (np.abs(lse[b] - l) <= e + (n + 16) * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(l))).all(), b


@pytest.mark.parametrize("listed", [False, True])
def test_segments_of_more_than_32_tiles(listed):
    # one request of 40 tiles for every SM and a part of one, over the same 8 pages again and again (or, listed, 1,024
    # requests' worth of spans over them): the walk looks pages up 32 tiles at a time
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pages = 8
    if listed:
        B, nsel = 40 * sms // 512 + 1, 1024
        lens = [256 * pages] * B
        cache, one = U.paged([256 * pages], seed=21)
        table = np.tile(one, (B, 1))
        spans = np.random.default_rng(21).integers(0, 4 * pages, (B, nsel)).astype(np.int32)
        tiles = B * nsel // 2
        counts = [np.repeat(np.bincount(s, minlength=4 * pages), 64) for s in spans]
    else:
        B, n = 1, 40 * 128 * sms + 77
        cache, one = U.paged([256 * pages], seed=21)
        table = np.tile(one, (1, -(-n // (256 * pages))))[:, :-(-n // 256)]
        lens, spans, tiles = [n], None, -(-n // 128)
        counts = [np.bincount(np.arange(n) % (256 * pages), minlength=256 * pages)]
    assert _tiles_per_cta(tiles) > 32
    qb = _queries(B, 21)
    ws = _workspace(B)
    out, lse = smla.decode_spans(U.dev_bf16(qb), U.dev(cache), U.dev(np.ascontiguousarray(table)), U.dev(np.array(lens, np.int32)), SCALE,
                                 spans=None if spans is None else U.dev(spans), workspace=ws)
    assert smla.read_error(ws) == 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    k = U.latents(cache, table, 0, np.arange(256 * pages))
    q = independent.q_values(qb)
    size = max(SCALE * float((np.abs(q[b]) @ np.abs(k).T).max()) for b in range(B))
    e = 512 * 2.0 ** -23 * size + 2.0 ** -21
    adds = _tiles_per_cta(tiles) * 128 + sms + 16  # a CTA's own tokens, then the parts
    for b in range(B):
        s = SCALE * (q[b] @ k.T)
        p = counts[b] * np.exp(s - s.max(axis=1, keepdims=True))
        total = p.sum(axis=1, keepdims=True)
        o, l, mean_abs = p @ k / total, (s.max(axis=1, keepdims=True) + np.log(total))[:, 0], p @ np.abs(k) / total
        off = np.abs(out[b] - o)
        bound = mean_abs * (2.0 ** -8 * (1 + 2 * e) + 2 * e + adds * 2.0 ** -23) + 2.0 ** -8 * (np.abs(o) + off)
        assert (off <= bound).all(), (b, float((off / bound).max()))
        assert (np.abs(lse[b] - l) <= e + adds * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(l))).all(), b


@pytest.mark.parametrize("lens", [[40000], [9000, 300, 17000, 1]])
def test_long_sequences_in_the_norm(lens):
    # Beside the element-wise bound: weights and outputs are each off by a rounding of rms 2^-8 / sqrt(3) at most,
    # independent from token to token; over latents of mean zero both are that share of the norm, together
    # 2^-8 sqrt(2 / 3) = 3.2e-3, below 4e-3
    out, _ = _run(lens, seed=22)
    cache, table = U.paged(lens, 22)
    q = independent.q_values(_queries(len(lens), 22))
    got = out.double().cpu().numpy()
    for b, n in enumerate(lens):
        want = U.attention(q[b], cache, table, b, np.arange(n), SCALE)[0]
        assert np.linalg.norm(got[b] - want) <= 4e-3 * np.linalg.norm(want), b


def test_captured_behind_two_streams_and_without_a_workspace():
    # a capture where the call's kernels follow work of two streams, and one where the workspace is allocated inside
    lens = np.array([3000, 700], np.int32)
    cache, table = U.paged(lens, seed=25)
    q, c, t, sl = U.dev_bf16(_queries(2, 25)), U.dev(cache), U.dev(table), U.dev(lens)
    keys = torch.zeros((len(cache), 4, 512), dtype=torch.bfloat16, device="cuda")
    keys.normal_(generator=torch.Generator("cuda").manual_seed(5))
    want = smla.decode_spans(q, c, t, sl, SCALE)
    want_scores = smla.span_scores(q, keys, t, sl, SCALE)
    ws, ws2 = _workspace(2), torch.zeros(smla.span_scores_workspace_bytes(*t.shape), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for given in (True, False):
        a, b = torch.zeros_like(q), torch.zeros_like(sl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            main, side = torch.cuda.current_stream(), torch.cuda.Stream()
            side.wait_stream(main)
            a.copy_(q)
            with torch.cuda.stream(side):
                b.copy_(sl)
                b.mul_(1)
            main.wait_stream(side)
            out, lse = smla.decode_spans(a, c, t, b, SCALE, workspace=ws if given else None)
            side.wait_stream(main)
            with torch.cuda.stream(side):
                b.add_(0)
            a.mul_(1)
            main.wait_stream(side)
            scores = smla.span_scores(a, keys, t, b, SCALE, workspace=ws2 if given else None)
        for _ in range(3):
            for x in (a, b, out, lse, scores):
                x.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(scores, want_scores)


def test_more_requests_than_threads_of_a_cta():
    # the lengths of two or three requests a thread, nine of ten of them empty, summed by every CTA and written out for the join
    rng = np.random.default_rng(28)
    lens = list(np.where(rng.random(2000) < 0.1, rng.integers(1, 140, 2000), rng.integers(-1, 1, 2000)))
    lens[0], lens[897], lens[1999] = 0, 1500, 129
    _run(lens, seed=28)


def test_pages_behind_4_gib():
    # a pool of 5.3 GB, the requests in its last pages; spans read, scored and attended there
    lens = [1000, 513]
    cache, table = U.paged(lens, seed=29)
    pages, first = 35500, 35500 - len(cache)
    assert first * W.PAGE_BYTES > 1 << 32
    pool = torch.empty((pages, W.PAGE_BYTES), dtype=torch.uint8, device="cuda")
    pool[first:] = U.dev(cache)
    far = np.where(table >= 0, table + first, -1).astype(np.int32)
    qb = _queries(2, 29)
    sl, ws = U.dev(np.array(lens, np.int32)), _workspace(2)
    out, lse = smla.decode_spans(U.dev_bf16(qb), pool, U.dev(far), sl, SCALE, workspace=ws)
    assert smla.read_error(ws) == 0
    U.check_decode(out, lse, independent.q_values(qb), cache, table, [np.arange(n) for n in lens], SCALE)
    req = np.repeat(np.arange(2), lens).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    for p, t in ((pool, far), (U.dev(cache), table)):
        rows = smla.read_kv(p, U.dev(req), U.dev(pos), U.dev(t), out_dtype=torch.float32)
        keys = torch.zeros((p.shape[0], 4, 512), dtype=torch.bfloat16, device="cuda")
        spans = [np.arange(-(-n // 64)) for n in lens]
        smla.span_keys(p, U.dev(t), sl, U.dev(np.repeat(np.arange(2), [len(s) for s in spans]).astype(np.int32)),
                       U.dev(np.concatenate(spans).astype(np.int32)), keys)
        got = (rows, keys[-len(cache):].clone(), smla.span_scores(U.dev_bf16(qb), keys, U.dev(t), sl, SCALE))
        if p is pool:
            want = got
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.isnan(got[0]).any() and got[1].any()


def test_keys_behind_4_gib():
    # 1.1 million pages of keys (4.5 GB): a request's last ones score as those of a small pool
    lens, pages = [9000, 300], 1_100_000
    rng = np.random.default_rng(30)
    table = rng.permutation(40)[:36 * 1].astype(np.int32)
    table = np.stack([table, np.r_[np.setdiff1d(np.arange(40), table)[:2], np.full(34, -1)]]).astype(np.int32)
    small = torch.randn((40, 4, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(30)).to(torch.bfloat16)
    pool = torch.empty((pages, 4, 512), dtype=torch.bfloat16, device="cuda")
    pool[-40:] = small
    far = np.where(table >= 0, table + pages - 40, -1).astype(np.int32)
    q, sl = U.dev_bf16(_queries(2, 30)), U.dev(np.array(lens, np.int32))
    assert torch.equal(smla.span_scores(q, pool, U.dev(far), sl, SCALE), smla.span_scores(q, small, U.dev(table), sl, SCALE))


def test_two_graphs_at_once_and_stream_handles():
    # graphs with a workspace each, replayed on two streams at the same time; streams given as plain handles
    lens = [[3000, 500, 41], [20000]]
    args, want, keys, want_scores = [], [], [], []
    for i, n in enumerate(lens):
        cache, table = U.paged(n, seed=31 + i)
        args.append((U.dev_bf16(_queries(len(n), 31 + i)), U.dev(cache), U.dev(table), U.dev(np.array(n, np.int32)), SCALE))
        keys.append(torch.randn((len(cache), 4, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(torch.bfloat16))
        want.append(smla.decode_spans(*args[i]))
        want_scores.append(smla.span_scores(args[i][0], keys[i], *args[i][2:]))
    torch.cuda.synchronize()
    graphs, got, spaces, streams = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        spaces.append((_workspace(len(lens[i])), torch.zeros(smla.span_scores_workspace_bytes(*args[i][2].shape), dtype=torch.uint8, device="cuda")))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            scores = smla.span_scores(args[i][0], keys[i], *args[i][2:], workspace=spaces[i][1])
            got.append((*smla.decode_spans(*args[i], workspace=spaces[i][0]), scores))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], (*want[i], want_scores[i])):
            assert torch.equal(a, b)
    for handle in (0, streams[0].cuda_stream):
        out = smla.decode_spans(*args[0], stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[1], want[0][1])
