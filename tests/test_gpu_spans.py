"""Reading the cache back, span keys and span selection through the binding, against 64-bit forms
(needs a B200).  The caches are NaN bytes wherever no request has a token.
"""
import numpy as np
import pytest
import torch

import sparse_mla_decode_fp8_b200 as smla
from sparse_mla_decode_fp8_b200 import build
from sparse_mla_decode_fp8_b200 import workloads as W
from tests import span_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    build.build()
    smla.library()


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- read_kv
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 31, 33, 257, 1000])
def test_read_kv_values_are_exact(dtype, n):
    lens = [700, 1, 300]
    cache, table = U.paged(lens, seed=n)
    rng = np.random.default_rng(n)
    req = rng.integers(0, 3, n).astype(np.int32)
    pos = (rng.random(n) * np.array(lens)[req]).astype(np.int32)
    err = _err()
    got = smla.read_kv(U.dev(cache), U.dev(req), U.dev(pos), U.dev(table), out_dtype=dtype, err=err)
    want = np.stack([U.latents(cache, table, b, [p])[0] for b, p in zip(req, pos)])
    # e4m3 * 2^e has 4 significant bits and lies far inside the bf16 range here: exact in both types
    assert got.dtype == dtype and np.array_equal(got.double().cpu().numpy(), want)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_kv_every_scale_byte(dtype):
    # token t of page 0 has scale bytes t in groups 0..5 and 255 - t in group 6; every e4m3 code occurs
    cache = np.zeros((1, W.PAGE_BYTES), np.uint8)
    rows, scales = W.row_views(cache)
    rows[0, :, :448] = np.arange(448)[None, :] % 256
    rows[0, :, 448:] = np.random.default_rng(3).integers(0, 256, (256, 128))
    scales[0, :, :6] = np.arange(256)[:, None]
    scales[0, :, 6] = 255 - np.arange(256)
    t = np.arange(256, dtype=np.int32)
    got = smla.read_kv(U.dev(cache), U.dev(np.zeros(256, np.int32)), U.dev(t), U.dev(np.zeros((1, 1), np.int32)),
                       out_dtype=dtype)
    want64 = torch.from_numpy(U.latents(cache, np.zeros((1, 1), np.int32), 0, t))
    want = want64.to(torch.float32).to(dtype)  # fp32 holds every product; beyond its range an infinity
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def test_read_kv_out_of_range_tokens_are_zero_rows():
    cache, table = U.paged([300, 300], seed=5)
    table[1, 1] = 99  # not a page
    req = np.array([0, -1, 2, 0, 0, 1, 0], np.int32)
    pos = np.array([299, 0, 0, -1, 512, 256, 0], np.int32)
    err = _err()
    out = torch.full((9, 512), 7.0, device="cuda")
    got = smla.read_kv(U.dev(cache), U.dev(req), U.dev(pos), U.dev(table), out=out[:7], err=err).double().cpu().numpy()
    assert np.array_equal(got[0], U.latents(cache, table, 0, [299])[0])
    assert np.array_equal(got[6], U.latents(cache, table, 0, [0])[0])
    assert not got[1:6].any()
    assert int(err.item()) == smla.SMLA_FLAG_BAD_PAGE
    assert (out[7:] == 7.0).all()  # rows behind the last token are left
    # without an error word, and with no token at all
    smla.read_kv(U.dev(cache), U.dev(req), U.dev(pos), U.dev(table), out=out[:7])
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert smla.read_kv(U.dev(cache), e, e, U.dev(table)).shape == (0, 512)


def test_write_then_read_back():
    # what the writer stores comes back within half an e4m3 step of its group's scale
    cache, table = U.paged([600], seed=6, garbage=False)
    x = torch.randn((600, 512), generator=torch.Generator().manual_seed(1))
    req, pos = np.zeros(600, np.int32), np.arange(600, dtype=np.int32)
    c, r, p, t = U.dev(cache), U.dev(req), U.dev(pos), U.dev(table)
    smla.write_kv(x.cuda(), r, p, t, c)
    got = smla.read_kv(c, r, p, t, out_dtype=torch.float32).cpu()
    top = x[:, :448].unflatten(1, (7, 64)).abs().amax(2, keepdim=True)
    # half a step: 2^-4 of the value, or half the subnormal step 2^-10 * 2^e with 2^e < top / 224
    bound = torch.maximum(x[:, :448].unflatten(1, (7, 64)).abs() * 2.0 ** -4, top / 224 * 2.0 ** -10)
    assert ((got[:, :448] - x[:, :448]).unflatten(1, (7, 64)).abs() <= bound).all()
    assert torch.equal(got[:, 448:], x[:, 448:].to(torch.bfloat16).float())


# ---------------------------------------------------------------- span_keys
@pytest.mark.parametrize("length", [1, 7, 63, 64, 65, 128, 255, 256, 257, 1000])
def test_span_keys_of_every_span(length):
    lens = np.array([length, 77], np.int32)
    cache, table = U.paged(lens, seed=length)
    req = np.concatenate([np.full(-(-n // 64), b) for b, n in enumerate(lens)]).astype(np.int32)
    span = np.concatenate([np.arange(-(-n // 64)) for n in lens]).astype(np.int32)
    keys = torch.full((len(cache), 4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    got = smla.span_keys(U.dev(cache), U.dev(table), U.dev(lens), U.dev(req), U.dev(span), keys, err=err)
    assert got is keys and int(err.item()) == 0
    got = got.double().cpu().numpy()
    touched = np.zeros(got.shape[:2], bool)
    for b, j in zip(req, span):
        want = U.span_mean(cache, table, lens, b, j)
        mean_abs = np.abs(U.latents(cache, table, b, np.arange(64 * j, min(64 * j + 64, lens[b])))).mean(axis=0)
        # fp32: at most 10 + 6 additions and one division, 2^-24 each of at most the sum of |x| / n;
        # then half a bf16 step, 2^-8 of the value
        bound = 2.0 ** -8 * np.abs(want) + 18 * 2.0 ** -24 * mean_abs
        assert (np.abs(got[table[b, j // 4], j % 4] - want) <= bound).all(), (b, j)
        touched[table[b, j // 4], j % 4] = True
    assert (got[~touched] == 3.0).all()  # the other keys are left as they were


def test_span_keys_skips_and_repeats():
    lens = np.array([130, 0, 512], np.int32)
    cache, table = U.paged(lens, seed=9)
    table[2, 1] = -1
    req = np.array([0, 0, 0, 1, 3, -1, 2, 0, 2], np.int32)
    span = np.array([2, 2, 3, 0, 0, 0, 4, -1, 1 << 20], np.int32)
    keys = torch.full((len(cache), 4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    smla.span_keys(U.dev(cache), U.dev(table), U.dev(lens), U.dev(req), U.dev(span), keys, err=err)
    got = keys.double().cpu().numpy()
    want = U.span_mean(cache, table, lens, 0, 2)
    assert (np.abs(got[table[0, 0], 2] - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()
    got[table[0, 0], 2] = 3.0
    assert (got == 3.0).all()
    assert int(err.item()) == smla.SMLA_FLAG_BAD_PAGE
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    smla.span_keys(U.dev(cache), U.dev(table), U.dev(lens), e, e, keys)


# ---------------------------------------------------------------- select_spans
def _select_case(width, kind, seed):
    rng = np.random.default_rng(seed)
    lens = np.array([64 * width, 64 * width - 1, max(1, 64 * (width // 2) - 5), 1, 0, -3, 64 * width + 999, 65], np.int32)
    x = rng.standard_normal((len(lens), width)).astype(np.float32)
    if kind == "ties":
        x = np.round(x * 2) / 2 * np.float32(0.25)
    elif kind == "equal":
        x[:] = 0.5
    elif kind == "special":
        x[rng.random(x.shape) < 0.2] = -np.inf
        x[rng.random(x.shape) < 0.1] = np.nan
        x[rng.random(x.shape) < 0.05] = np.inf
        x[rng.random(x.shape) < 0.2] = 0.0
        x[rng.random(x.shape) < 0.2] = -0.0
        x[rng.random(x.shape) < 0.1] = np.float32(1e-42)
        x[0] = np.nan
        x[1] = -np.inf
        x[2] = np.finfo(np.float32).min
    elif kind == "negative":
        x = -np.abs(x)
    return x, lens


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special", "negative"])
@pytest.mark.parametrize("width", [1, 2, 5, 64, 257, 2048, 2049, 8192, 8193, 9000])
def test_select_spans_equals_sorting(width, kind):
    x, lens = _select_case(width, kind, seed=width)
    for nsel, first, last in [(1, 0, 0), (1, 1, 0), (3, 1, 2), (8, 1, 1), (33, 0, 2), (1024, 4, 3)]:
        spans, idx = smla.select_spans(U.dev(x), U.dev(lens), nsel, keep_first=first, keep_last=last)
        want_spans, want_idx = U.select(x, lens, nsel, first, last)
        assert np.array_equal(spans.cpu().numpy(), want_spans), (nsel, first, last)
        assert np.array_equal(idx.cpu().numpy(), want_idx), (nsel, first, last)


@pytest.mark.parametrize("width", [4096, 4097, 16384, 16385, 40000])
def test_select_spans_of_long_rows(width):
    for kind in ("random", "special"):
        x, lens = _select_case(width, kind, seed=width)
        for nsel, first, last in [(1, 0, 0), (33, 1, 2), (1024, 4, 3)]:
            spans, idx = smla.select_spans(U.dev(x), U.dev(lens), nsel, keep_first=first, keep_last=last)
            want_spans, want_idx = U.select(x, lens, nsel, first, last)
            assert np.array_equal(spans.cpu().numpy(), want_spans) and np.array_equal(idx.cpu().numpy(), want_idx)


def test_select_spans_without_tokens_and_into_given_tensors():
    x, lens = _select_case(100, "random", 1)
    spans = torch.full((len(lens), 7), 55, dtype=torch.int32, device="cuda")
    got, idx = smla.select_spans(U.dev(x), U.dev(lens), 7, spans=spans, tokens=False)
    assert got is spans and idx is None
    assert np.array_equal(spans.cpu().numpy(), U.select(x, lens, 7, 0, 0)[0])
    # the list is what the sparse decode takes
    spans, idx = smla.select_spans(U.dev(x), U.dev(lens), 7)
    assert idx.shape == (len(lens), 7 * 64) and idx.dtype == torch.int32


def test_select_spans_on_another_stream_and_in_a_graph():
    x, lens = _select_case(300, "ties", 2)
    dx, dl = U.dev(x), U.dev(lens)
    want = U.select(x, lens, 5, 1, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spans, idx = smla.select_spans(dx, dl, 5, keep_first=1, keep_last=1, stream=side)
    side.synchronize()
    assert np.array_equal(spans.cpu().numpy(), want[0]) and np.array_equal(idx.cpu().numpy(), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spans, idx = smla.select_spans(dx, dl, 5, keep_first=1, keep_last=1)
    y, _ = _select_case(300, "random", 3)
    dx.copy_(U.dev(y))
    g.replay()
    torch.cuda.synchronize()
    want = U.select(y, lens, 5, 1, 1)
    assert np.array_equal(spans.cpu().numpy(), want[0]) and np.array_equal(idx.cpu().numpy(), want[1])


def test_span_keys_of_lists_longer_than_the_grid():
    # about five spans a block: full, partial and skipped ones in any order, some listed again
    lens = np.array([5000, 63, 1, 4097, 640, 2222, 0, 130], np.int32)
    cache, table = U.paged(lens, seed=26)
    table[4, 1] = -1
    n = 5 * 4 * torch.cuda.get_device_properties(0).multi_processor_count + 37
    rng = np.random.default_rng(26)
    req = rng.integers(-1, len(lens) + 1, n).astype(np.int32)
    have = np.array([-(-max(int(x), 0) // 64) for x in lens])
    span = np.where(rng.random(n) < 0.2, rng.integers(-3, 200, n), (rng.random(n) * have[req % len(lens)]).astype(np.int64)).astype(np.int32)
    last = rng.random(n) < 0.2  # the partial ones more often
    span[last] = (have[req % len(lens)] - 1)[last]
    keys = torch.full((len(cache), 4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    smla.span_keys(U.dev(cache), U.dev(table), U.dev(lens), U.dev(req), U.dev(span), keys, err=err)
    assert int(err.item()) == smla.SMLA_FLAG_BAD_PAGE
    got = keys.double().cpu().numpy()
    touched = np.zeros(got.shape[:2], bool)
    live = 0
    for b, j in set(zip(req.tolist(), span.tolist())):
        if not (0 <= b < len(lens) and 0 <= j < have[b]) or table[b, j // 4] < 0:
            continue
        live += 1
        want = U.span_mean(cache, table, lens, b, j)
        mean_abs = np.abs(U.latents(cache, table, b, np.arange(64 * j, min(64 * j + 64, lens[b])))).mean(axis=0)
        bound = 2.0 ** -8 * np.abs(want) + 18 * 2.0 ** -24 * mean_abs  # as for single spans
        assert (np.abs(got[table[b, j // 4], j % 4] - want) <= bound).all(), (b, j)
        touched[table[b, j // 4], j % 4] = True
    assert live > 150 and (got[~touched] == 3.0).all()
