"""The span operators at the largest sizes their header allows (needs a B200)."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_fp8_b200 as smla
from sparse_mla_decode_fp8_b200 import build
from tests import span_util as U

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
MAX_SPANS = 1 << 25


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    build.build()
    smla.library()


@pytest.mark.parametrize("nsel,first,last", [(7, 1, 1), (1024, 0, 0)])
def test_select_from_the_most_spans(nsel, first, last):
    # scores all different, made of consecutive fp32 bit patterns; the last token is number 2^31 - 2
    g = torch.Generator("cuda").manual_seed(1)
    order = torch.randperm(MAX_SPANS, generator=g, device="cuda", dtype=torch.int32)
    scores = (order + 0x3F000000).view(torch.float32).view(1, MAX_SPANS)
    spans, idx = smla.select_spans(scores, torch.tensor([2**31 - 1], dtype=torch.int32, device="cuda"), nsel, keep_first=first, keep_last=last)
    key = order.long()
    key[:first] += 1 << 40
    key[MAX_SPANS - last:] += 1 << 40
    want = torch.topk(key, nsel).indices.sort().values
    assert torch.equal(spans[0].long(), want)
    tokens = (want.unsqueeze(1) * 64 + torch.arange(64, device="cuda")).flatten()
    assert torch.equal(idx[0].long(), torch.where(tokens < 2**31 - 1, tokens, -1))


def test_the_widest_block_table():
    # 2^23 pages a request, all but two of them none; scores behind the last span are zeros
    lens = [500]
    cache, table = U.paged(lens, seed=2)
    wide = torch.full((1, MAX_SPANS // 4), -1, dtype=torch.int32, device="cuda")
    small = U.dev(table)
    wide[:, :small.shape[1]] = small
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.randn((1, 64, 512), generator=g, device="cuda").to(torch.bfloat16)
    keys = torch.randn((len(cache), 4, 512), generator=g, device="cuda").to(torch.bfloat16)
    sl, c = U.dev(np.array(lens, np.int32)), U.dev(cache)
    got, want = smla.span_scores(q, keys, wide, sl, SCALE), smla.span_scores(q, keys, small, sl, SCALE)
    assert torch.equal(got[:, :want.shape[1]], want) and not got[:, want.shape[1]:].any()
    for a, b in zip(smla.decode_spans(q, c, wide, sl, SCALE), smla.decode_spans(q, c, small, sl, SCALE)):
        assert torch.equal(a, b)


def test_the_most_requests():
    # 65,535 requests of up to 128 tokens (a tile, so that none is cut): some of them again in a small batch
    B = 65535
    cache, one = U.paged([256 * 8], seed=3)
    g = torch.Generator("cuda").manual_seed(3)
    pages = U.dev(one[0])
    table = pages[torch.randint(0, 8, (B, 1), generator=g, device="cuda")].contiguous()
    lens = torch.randint(-2, 129, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.empty((B, 64, 512), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    keys = torch.randn((len(cache), 4, 512), generator=g, device="cuda").to(torch.bfloat16)
    c = U.dev(cache)
    out, lse = smla.decode_spans(q, c, table, lens, SCALE)
    scores = smla.span_scores(q, keys, table, lens, SCALE)
    some = torch.cat([torch.arange(0, B, 1311, device="cuda"), torch.tensor([B - 1], device="cuda")])
    part = [x[some].contiguous() for x in (q, table, lens)]
    few, few_lse = smla.decode_spans(part[0], c, part[1], part[2], SCALE)
    assert torch.equal(out[some], few) and torch.equal(lse[some], few_lse)
    assert torch.equal(scores[some], smla.span_scores(part[0], keys, part[1], part[2], SCALE))
    # by the 64-bit form as well
    host = [x.cpu() for x in part]
    U.check_decode(few, few_lse, host[0].double().numpy(), cache, host[1].numpy(), [np.arange(max(int(n), 0)) for n in host[2]], SCALE)
    assert torch.isneginf(lse[lens <= 0]).all() and not out[lens <= 0].any()
