"""What the span operators and the cache reader refuse, without a GPU: the C entry points check
sizes, pointers and alignment before they look for a device, the binding checks its tensors."""
import ctypes

import pytest
import torch

import sparse_mla_decode_fp8_b200 as smla
from sparse_mla_decode_fp8_b200 import build

INVALID = -1
A, ODD, ODD16 = 1 << 20, (1 << 20) + 2, (1 << 20) + 8  # addresses that are never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return smla.library()


READ = [A, A, A, 5, A, 2, 3, 4, A, 1, A, None]
KEYS = [A, A, A, A, A, 5, 2, 3, 4, A, A, None]
DECODE = [A, A, A, None, 0, A, 0.1, A, A, 2, 64, 3, 4, A, 1 << 30, None, None]
SCORES = [A, A, A, A, 0.1, A, 2, 64, 3, 4, A, 1 << 30, None, None]
SELECT = [A, 100, A, 8, 1, 1, A, A, 2, None]


def _refused(fn, args, changes):
    for at, bad in changes:
        call = list(args)
        call[at] = bad
        assert fn(*call) == INVALID, (at, bad)


def test_read_kv_refuses(lib):
    _refused(lib.smla_read_kv, READ, [(0, None), (1, None), (2, None), (4, None), (8, None), (3, -1), (5, 0), (6, 0),
                                      (7, 0), (7, 1 << 23), (0, ODD16), (8, ODD16), (1, ODD), (2, ODD), (4, ODD), (10, ODD)])
    assert lib.smla_read_kv(None, None, None, 0, None, 1, 1, 1, None, 1, None, None) == 0  # nothing to read


def test_span_keys_refuses(lib):
    _refused(lib.smla_span_keys, KEYS, [(k, None) for k in (0, 1, 2, 3, 4, 9)] + [(5, -1), (6, 0), (7, 0), (8, 0),
             (8, 1 << 23), (0, ODD16), (9, ODD16), (1, ODD), (2, ODD), (3, ODD), (4, ODD), (10, ODD)])
    assert lib.smla_span_keys(None, None, None, None, None, 0, 1, 1, 1, None, None, None) == 0


def test_select_spans_refuses(lib):
    _refused(lib.smla_select_spans, SELECT, [(0, None), (2, None), (6, None), (1, 0), (1, (1 << 25) + 1), (3, 0), (3, 1025),
             (4, -1), (5, -1), (4, 8), (5, 8), (4, 2**31 - 1), (8, 0), (0, ODD), (2, ODD), (6, ODD), (7, ODD)])


def test_decode_spans_refuses(lib):
    _refused(lib.smla_decode_spans, DECODE, [(k, None) for k in (0, 1, 2, 5, 7, 8, 13)] + [(4, 3), (4, -1), (6, float("nan")),
             (6, float("inf")), (9, 0), (9, 65536), (10, 32), (11, 0), (12, 0), (12, 1 << 23), (0, ODD16), (1, ODD16),
             (7, ODD16), (13, A + 128), (2, ODD), (3, ODD), (5, ODD), (8, ODD)])
    listed = DECODE[:3] + [A] + DECODE[4:]
    _refused(lib.smla_decode_spans, listed, [(4, 0), (4, 1025)])
    for nsplit, out_bf16 in ((2, 1), (0, 0)):
        opts = smla.binding._Options(nsplit, out_bf16, 0, 0, 0)
        _refused(lib.smla_decode_spans, DECODE, [(15, ctypes.byref(opts))])
    assert lib.smla_decode_spans_workspace_bytes(0) == 0 and lib.smla_decode_spans_workspace_bytes(65536) == 0


def test_span_scores_refuses(lib):
    _refused(lib.smla_span_scores, SCORES, [(k, None) for k in (0, 1, 2, 3, 5, 10)] + [(4, float("nan")), (6, 0), (6, 65536),
             (7, 32), (8, 0), (8, (1 << 23) + 1), (9, 0), (9, 1 << 23), (0, ODD16), (1, ODD16), (10, A + 128), (2, ODD),
             (3, ODD), (5, ODD), (11, 1000)])
    for nsplit, out_bf16 in ((2, 0), (0, 1)):
        opts = smla.binding._Options(nsplit, out_bf16, 0, 0, 0)
        _refused(lib.smla_span_scores, SCORES, [(12, ctypes.byref(opts))])
    assert lib.smla_span_scores_workspace_bytes(0, 5) == 0 and lib.smla_span_scores_workspace_bytes(5, 0) == 0
    # header, 2 tiles of 64 (maximum, sum) per request, 64 fp32 per span
    assert lib.smla_span_scores_workspace_bytes(3, 40) == 256 + 3 * 2 * 64 * 8 + 3 * 160 * 64 * 4


def test_binding_refuses_host_tensors():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(smla.SmlaError):
        smla.read_kv(torch.zeros((1, 149504), dtype=torch.uint8), i, i, i.view(1, 3))
    with pytest.raises(smla.SmlaError):
        smla.span_keys(torch.zeros((1, 149504), dtype=torch.uint8), i.view(1, 3), i[:1], i, i,
                       torch.zeros((1, 4, 512), dtype=torch.bfloat16))
    with pytest.raises(smla.SmlaError):
        smla.select_spans(torch.zeros((3, 8)), i, 2)


def test_entry_points_take_their_argument_counts(lib):
    # every argument is described to ctypes: a call with one missing raises instead of running
    for fn, args in ((lib.smla_read_kv, READ), (lib.smla_span_keys, KEYS), (lib.smla_select_spans, SELECT),
                     (lib.smla_decode_spans, DECODE), (lib.smla_span_scores, SCORES)):
        assert len(fn.argtypes) == len(args)
        with pytest.raises((TypeError, ctypes.ArgumentError)):
            fn(*args[:-1])


def test_binding_refuses_numbers_beyond_the_abi_types(monkeypatch):
    # ctypes would take them modulo 2^32 (2^64) and run with another number
    monkeypatch.setattr(smla.binding, "_current", lambda t, name: 0)

    def meta(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")

    wide = 2**32 + 5
    cache, keys, one = meta(1, 149504, dtype=torch.uint8), meta(1, 4, 512, dtype=torch.bfloat16), meta(1, 1)
    q, f32 = meta(1, 64, 512, dtype=torch.bfloat16), torch.float32
    calls = [lambda: smla.select_spans(meta(1, wide, dtype=f32), meta(1), 2), lambda: smla.select_spans(meta(wide, 1, dtype=f32), meta(wide), 2),
             lambda: smla.span_keys(cache, one, meta(1), meta(wide), meta(wide), keys), lambda: smla.read_kv(cache, meta(wide), meta(wide), one)]
    for first, last in ((2**32, 0), (0, 2**32), (2**32 + 1, 1), (-(2**32), 0), (-1, 0), (1, 2), (3, 0)):
        calls.append(lambda first=first, last=last: smla.select_spans(meta(1, 8, dtype=f32), meta(1), 2, keep_first=first, keep_last=last))
    for kw in (dict(wait_timeout_ns=-1), dict(wait_timeout_ns=2**64), dict(debug_flags=2**32), dict(debug_flags=-1)):
        calls += [lambda kw=kw: smla.decode_spans(q, cache, one, meta(1), 0.1, **kw), lambda kw=kw: smla.span_scores(q, keys, one, meta(1), 0.1, **kw)]
    for i, call in enumerate(calls):
        with pytest.raises(smla.SmlaError, match="must"):
            call()
