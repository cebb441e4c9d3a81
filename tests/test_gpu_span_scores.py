"""smla_span_scores through the binding against 64-bit softmaxes, and the operators in a row as a decode
step uses them (needs a B200)."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_fp8_b200 as smla
from sparse_mla_decode_fp8_b200 import build
from sparse_mla_decode_fp8_b200 import workloads as W
from tests import independent
from tests import span_util as U

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    build.build()
    smla.library()


def _case(lens, seed, size=0.5):
    """(q bits, key bits [pages, 4, 512], table); keys that no request has are NaN."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-max(int(n), 0) // 256)) for n in lens]
    pages = sum(need) + 2
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(need)), -1, np.int32)
    keys = np.full((pages, 4, 512), np.nan, np.float32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
        j = np.arange(-(-max(int(lens[b]), 0) // 64))
        keys[table[b, j // 4], j % 4] = size * rng.standard_normal((len(j), 512))
    q = W.to_bf16_bits(rng.standard_normal((len(lens), 64, 512)).astype(np.float32))
    return q, W.to_bf16_bits(keys), table


def _workspace(B, blocks):
    ws = torch.full((smla.span_scores_workspace_bytes(B, blocks),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    return ws


def _check(got, q, keys, table, lens, sm_scale):
    """A score is a sum over 64 heads of p = e^(x - lambda).  x: 512 exact products added in fp32, at most 2^-23
    of the largest partial sum each, and two more roundings of |x|; lambda carries the same and n + 80
    additions; so |dp| <= p (2 dx + (n + 80) 2^-23 + 2^-20), and the sum over the heads as much."""
    qv, kv = independent.q_values(q), independent.q_values(keys)
    want = U.scores(qv, kv, table, lens, sm_scale)
    got = got.double().cpu().numpy()
    for b, n in enumerate(lens):
        j = np.arange(min(-(-max(int(n), 0) // 64), 4 * table.shape[1]))
        page = table[b, j // 4]
        j = j[(page >= 0) & (page < len(kv))]
        size = abs(sm_scale) * float((np.abs(qv[b]) @ np.abs(kv[table[b, j // 4], j % 4]).T).max()) if len(j) else 0.0
        rel = 2 * (512 * 2.0 ** -23 + 2.0 ** -22) * size + (len(j) + 80) * 2.0 ** -23 + 2.0 ** -20
        off = np.abs(got[b] - want[b])
        assert (off <= rel * want[b] + 1e-37).all(), (b, float((off / np.maximum(want[b], 1e-37)).max()), rel)
        assert not got[b, -(-max(int(n), 0) // 64):].any()


def _run(lens, seed, sm_scale=SCALE, size=0.5, **kw):
    q, keys, table = _case(lens, seed, size)
    ws = _workspace(len(lens), table.shape[1])
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.asarray(lens, np.int32)), sm_scale,
                           workspace=ws, **kw)
    torch.cuda.synchronize()
    assert smla.read_error(ws) == 0
    _check(got, q, keys, table, lens, sm_scale)
    return got


@pytest.mark.parametrize("length", [1, 64, 65, 8191, 8192, 8193, 20000])
def test_one_request(length):
    _run([length], seed=length)


@pytest.mark.parametrize("lens", [[0], [0, 0, 100, 0], [-5, 700], [9000, 0, 1, 64, 30000, 129]])
def test_ragged(lens):
    got = _run(lens, seed=len(lens))
    for b, n in enumerate(lens):  # 64 softmaxes
        assert abs(float(got[b].double().sum()) - (64 if n > 0 else 0)) <= 1e-4


def test_more_tiles_than_ctas():
    _run(list(np.random.default_rng(1).integers(0, 40000, 120)), seed=1)


def test_more_requests_than_ctas():
    _run(list(np.random.default_rng(2).integers(0, 3000, 300)), seed=2)


@pytest.mark.parametrize("sm_scale,size", [(0.0, 0.5), (-SCALE, 0.5), (1.0, 2.0)])
def test_scales(sm_scale, size):
    _run([5000, 700], seed=4, sm_scale=sm_scale, size=size)


def test_bad_pages_take_no_part():
    lens = [1000, 300, 600]
    q, keys, table = _case(lens, 5)
    table[0, 1], table[1, :] = len(keys), -1
    ws = _workspace(3, table.shape[1])
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE, workspace=ws)
    assert smla.read_error(ws) == smla.SMLA_FLAG_BAD_PAGE
    _check(got, q, keys, table, lens, SCALE)
    assert not got[1].any() and not got[0, 4:8].any()


def test_repeats_on_a_stream_in_a_graph_and_into_a_given_tensor():
    lens = np.array([9000, 333], np.int32)
    q, keys, table = _case([20000, 20000], 6)
    args = [U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(lens)]
    out = torch.full((3, 4 * table.shape[1]), 7.0, device="cuda")
    first = smla.span_scores(*args, SCALE, scores=out[:2]).clone()
    _check(first, q, keys, table, lens, SCALE)
    assert (out[2] == 7.0).all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = smla.span_scores(*args, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(again, first)
    ws = _workspace(2, table.shape[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = smla.span_scores(*args, SCALE, workspace=ws)
    for lens in ([20000, 0], [65, 12345]):
        args[3].copy_(U.dev(np.array(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        _check(got, q, keys, table, lens, SCALE)


@pytest.mark.parametrize("lens", [[100], [30000, 50, 0], [40000] * 20])
def test_a_wait_that_runs_out_is_reported_and_leaves_nan_scores(lens):
    q, keys, table = _case(lens, 7)
    args = (U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    ws = _workspace(len(lens), table.shape[1])
    got = smla.span_scores(*args, workspace=ws, wait_timeout_ns=2_000_000, debug_flags=smla.SMLA_DEBUG_SKIP_FIRST_COMMIT)
    torch.cuda.synchronize()
    assert smla.read_error(ws) & smla.SMLA_FLAG_TIMEOUT
    for b, n in enumerate(lens):
        spans = -(-n // 64)
        assert torch.isnan(got[b, :spans]).all() and not got[b, spans:].any()
    got = smla.span_scores(*args, workspace=ws)
    assert smla.read_error(ws) == 0
    _check(got, q, keys, table, lens, SCALE)


def test_refusals():
    q, keys, table = _case([300], 8)
    q, k, t, l = U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array([300], np.int32))
    for args in ((q[:, :32], k, t, l), (q, k[:, :3], t, l), (q, k, t[0], l), (q, k, t, l.long()), (q.cpu(), k, t, l), (q, k.float(), t, l)):
        with pytest.raises(smla.SmlaError):
            smla.span_scores(*args, SCALE)
    for bad in (dict(scores=torch.empty((1, 7), device="cuda")), dict(workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(smla.SmlaError):
            smla.span_scores(q, k, t, l, SCALE, **bad)
    with pytest.raises(smla.SmlaError):
        smla.span_scores(q, k, t, l, float("inf"))


def test_nan_in_a_query_or_a_key_stays_with_its_request():
    lens = [9000, 500, 700]
    q, keys, table = _case(lens, 10)
    args = (U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    ref = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), *args)
    q[0, 3, 9] = 0x7FC0
    keys[table[1, 0], 2, 17] = 0x7FC0
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), *args)
    for b in (0, 1):
        n = -(-lens[b] // 64)
        assert torch.isnan(got[b, :n]).all() and not got[b, n:].any()
    assert torch.equal(got[2], ref[2])


def test_empty_requests_alone_and_calls_back_to_back_on_one_workspace():
    # nothing but empty requests, then work, then nothing again, without a wait between the calls
    q, keys, table = _case([20000, 20000], 11)
    a = [U.dev_bf16(q), U.dev_bf16(keys), U.dev(table)]
    lens = [[0, -4], [20000, 1], [0, 0], [8200, 20000]]
    ws = _workspace(2, table.shape[1])
    sl = [U.dev(np.array(n, np.int32)) for n in lens]
    got = [smla.span_scores(*a, x, SCALE, workspace=ws) for x in sl]
    torch.cuda.synchronize()
    for g, n in zip(got, lens):
        _check(g, q, keys, table, n, SCALE)


def test_two_calls_at_once_with_a_workspace_each():
    calls = []
    for seed, lens in ((12, [20000, 3000]), (13, [64] * 40)):
        q, keys, table = _case(lens, seed)
        calls.append((U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE))
    want = [smla.span_scores(*c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [_workspace(*c[2].shape) for c in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, st, ws in zip(calls, streams, spaces):
            got.append(smla.span_scores(*c, workspace=ws, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


def test_inputs_rewritten_right_before_each_call():
    # lengths, queries, cache rows and keys change on the stream between the calls, with and without waits for the GPU:
    # the calls start while the kernels before them drain, and must not see what those have yet to write
    rng = np.random.default_rng(14)
    table = U.dev(rng.permutation(40).reshape(2, 20).astype(np.int32))
    base = torch.randn((2, 64, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    rows = torch.randn((30, 2, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    r = U.dev(np.arange(2, dtype=np.int32))
    ws, ws2 = _workspace(2, 20), torch.zeros(smla.decode_spans_workspace_bytes(2), dtype=torch.uint8, device="cuda")

    def steps(wait):
        cache = torch.zeros((40, W.PAGE_BYTES), dtype=torch.uint8, device="cuda")
        keys = torch.zeros((40, 4, 512), dtype=torch.bfloat16, device="cuda")
        lens, q, got = U.dev(np.array([100, 3000], np.int32)), torch.empty((2, 64, 512), dtype=torch.bfloat16, device="cuda"), []
        for i in range(30):
            lens.add_(1)
            q.copy_(base * (1 + i))
            smla.write_kv(rows[i], r, lens - 1, table, cache)
            smla.span_keys(cache, table, lens, r, (lens - 1) // 64, keys)
            scores = smla.span_scores(q, keys, table, lens, SCALE, workspace=ws)
            spans, _ = smla.select_spans(scores, lens, 5, keep_last=1)
            out, lse = smla.decode_spans(q, cache, table, lens, SCALE, spans=spans, workspace=ws2)
            whole = smla.decode_spans(q, cache, table, lens, SCALE, workspace=ws2)
            got.append((scores, spans, out, lse, *whole))
            lens.mul_(1)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got

    for x, y in zip(steps(True), steps(False)):
        for a, b in zip(x, y):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- the operators in a row
def test_a_decode_step_over_selected_spans():
    # prefill by the writer, keys of every span, then three steps: write a token, its span's key, scores,
    # selection, attention over it both ways; everything against 64 bits on what the cache then holds
    lens, nsel, B = np.array([2500, 640, 63], np.int32), 6, 3
    rng = np.random.default_rng(9)
    pages = 32
    table = rng.permutation(pages)[:30].reshape(B, 10).astype(np.int32)
    cache = torch.full((pages, W.PAGE_BYTES), 0xFF, dtype=torch.uint8, device="cuda")
    keys = torch.full((pages, 4, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    dt = U.dev(table)
    lat = torch.randn((int(lens.sum()), 512), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    req = np.repeat(np.arange(B), lens).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    smla.write_kv(lat, U.dev(req), U.dev(pos), dt, cache)
    back = smla.read_kv(cache, U.dev(req), U.dev(pos), dt, out_dtype=torch.float32)
    # half an e4m3 step is at most 2^-4 of a value in the normal range, 2^-10 of 448 scales below; rope 2^-8
    assert (back - lat).abs().max() <= 2.0 ** -4 * lat.abs().max()
    span = np.concatenate([np.arange(-(-n // 64)) for n in lens]).astype(np.int32)
    smla.span_keys(cache, dt, U.dev(lens), U.dev(np.repeat(np.arange(B), -(-lens // 64)).astype(np.int32)), U.dev(span), keys)
    for step in range(3):
        lens = lens + 1
        dl, r = U.dev(lens), U.dev(np.arange(B, dtype=np.int32))
        new = torch.randn((B, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(10 + step))
        smla.write_kv(new, r, dl - 1, dt, cache)
        smla.span_keys(cache, dt, dl, r, (dl - 1) // 64, keys)
        qb = W.to_bf16_bits(rng.standard_normal((B, 64, 512)).astype(np.float32))
        q = U.dev_bf16(qb)
        scores = smla.span_scores(q, keys, dt, dl, SCALE)
        spans, idx = smla.select_spans(scores, dl, nsel, keep_first=1, keep_last=1)
        out, lse = smla.decode_spans(q, cache, dt, dl, SCALE, spans=spans)
        sparse, sparse_lse = smla.decode(q, cache, dt, idx, dl, SCALE)
        host = cache.cpu().numpy()
        _check(scores, qb, keys.cpu().view(torch.int16).numpy().view(np.uint16), table, lens, SCALE)
        want_spans, want_idx = U.select(scores.cpu().numpy(), lens, nsel, 1, 1)
        assert np.array_equal(spans.cpu().numpy(), want_spans) and np.array_equal(idx.cpu().numpy(), want_idx)
        qv = independent.q_values(qb)
        U.check_decode(out, lse, qv, host, table, [want_idx[b][want_idx[b] >= 0] for b in range(B)], SCALE)
        U.check_decode(sparse, sparse_lse, qv, host, table, [want_idx[b][want_idx[b] >= 0] for b in range(B)], SCALE)


@pytest.mark.parametrize("spans", [127, 128, 129, 130, 192, 256, 257])
def test_a_nan_in_the_newest_key_reaches_every_span(spans):
    # alone in its tile or not, the NaN is in the sum of every head
    lens = [64 * spans - 63, 500]
    q, keys, table = _case(lens, 15)
    args = (U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    ref = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), *args)
    keys[table[0, (spans - 1) // 4], (spans - 1) % 4, 100] = 0x7FC0
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), *args)
    assert torch.isnan(got[0, :spans]).all() and not got[0, spans:].any()
    assert torch.equal(got[1], ref[1])


def test_keys_of_infinite_size():
    # scores of -inf beside others weigh nothing, alone in a tile or not; a request that has no others has no weight
    lens = [64 * 129, 64 * 20, 64 * 130]
    q, keys, table = _case(lens, 17)
    q[:, :, 9] = W.to_bf16_bits(np.ones(1, np.float32))
    low = W.to_bf16_bits(np.array([-np.inf], np.float32))[0]
    keys[table[0, 32], 0, 9] = low                     # span 128 of the first request
    keys[table[1, 1], 2, 9] = low                      # span 6 of the second
    for j in range(130):
        keys[table[2, j // 4], j % 4, 9] = low         # all of the third
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    assert got[0, 128] == 0 and got[1, 6] == 0
    for b, n in ((0, 129), (1, 20)):
        assert not torch.isnan(got[b]).any() and abs(float(got[b, :n].double().sum()) - 64) <= 1e-4
    assert not got[2].any()


def test_a_nan_between_bad_pages():
    # the NaN keys are the only ones of their tile; spans in bad pages score 0 whatever the others do
    lens = [64 * 256, 64 * 40]
    q, keys, table = _case(lens, 16)
    keys[table[0, 32], :, 5] = 0x7FC0
    table[0, 33:64] = -1
    table[1, 3] = len(keys)
    ws = _workspace(2, table.shape[1])
    got = smla.span_scores(U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE, workspace=ws)
    assert smla.read_error(ws) == smla.SMLA_FLAG_BAD_PAGE
    assert torch.isnan(got[0, :132]).all() and not got[0, 132:].any()
    assert not torch.isnan(got[1]).any() and not got[1, 12:16].any()


def test_calls_in_a_row_equal_calls_apart():
    # the steps above against a run that waits for the GPU before every single call: no kernel can start there before
    # what it reads is written
    rng = np.random.default_rng(18)
    table = U.dev(rng.permutation(600).reshape(2, 300).astype(np.int32))
    base = torch.randn((2, 64, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    fill = torch.randn((600, 4, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(9)).to(torch.bfloat16)
    steps = [np.array(x, np.int32) for x in ([76000, 100], [0, 0], [64, 76800], [9000, 9000], [1, 0], [40000, 76800], [0, 1], [8193, 64])]
    steps = [U.dev(x) for x in steps] * 3
    ws, ws2 = _workspace(2, 300), torch.zeros(smla.decode_spans_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    cache = torch.zeros((600, W.PAGE_BYTES), dtype=torch.uint8, device="cuda")
    rows = torch.randn((153600, 512), device="cuda", generator=torch.Generator("cuda").manual_seed(10))
    at = torch.arange(153600, dtype=torch.int32, device="cuda")
    smla.write_kv(rows, at // 76800, at % 76800, table, cache)

    def run(apart):
        def gap():
            if apart:
                torch.cuda.synchronize()
        lens, q, keys, got = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.empty_like(base, dtype=torch.bfloat16), fill.clone(), []
        for i, new in enumerate(steps):
            q.copy_(base * (1 + i))
            keys.copy_(fill * (1 + i % 3))
            lens.copy_(new)
            gap()
            scores = smla.span_scores(q, keys, table, lens, SCALE, workspace=ws)
            gap()
            lens.zero_()          # right behind the call: it has read its lengths by then
            lens.copy_(new)
            gap()
            spans, _ = smla.select_spans(scores, lens, 9, keep_last=1)
            gap()
            out, lse = smla.decode_spans(q, cache, table, lens, SCALE, spans=spans, workspace=ws2)
            gap()
            lens.fill_(3)
            gap()
            got.append((scores, spans, out, lse))
        torch.cuda.synchronize()
        return got

    for x, y in zip(run(True), run(False)):
        for a, b in zip(x, y):
            assert torch.equal(a, b)


@pytest.mark.parametrize("hook", [0, smla.SMLA_DEBUG_SKIP_FIRST_COMMIT])
@pytest.mark.parametrize("lens", [[100], [1000, 50, 0], [40000, 1, 300], [3000] * 200])
def test_a_limit_of_a_nanosecond(lens, hook):
    # shorter than any copy: a request is right or NaN, and the CTAs that gave up have waited for their copies and MMAs
    q, keys, table = _case(lens, 27)
    args = (U.dev_bf16(q), U.dev_bf16(keys), U.dev(table), U.dev(np.array(lens, np.int32)), SCALE)
    want = smla.span_scores(*args)
    for i in range(5):
        ws = _workspace(*table.shape)
        got = smla.span_scores(*args, workspace=ws, wait_timeout_ns=1, debug_flags=hook)
        torch.cuda.synchronize()
        flags = smla.read_error(ws)
        assert flags in (0, smla.SMLA_FLAG_TIMEOUT) and (flags or not hook)
        for b, n in enumerate(lens):
            spans = -(-n // 64)
            nan = bool(torch.isnan(got[b]).any())
            assert nan <= (flags != 0) and (nan or not hook or n <= 0)
            assert not got[b, spans:].any() and (torch.isnan(got[b, :spans]).all() if nan else torch.equal(got[b], want[b]))
    again = smla.span_scores(*args)
    assert torch.equal(again, want)
