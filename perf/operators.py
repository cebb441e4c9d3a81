"""The long-context operators beside the sparse decode, as measured cases.

Five operators over the FP8 paged latent cache (256-token pages: 256 rows of 448 e4m3 + 64 bf16 values, then
256 scale rows of 8 UE8M0 bytes).  A *span* is 64 consecutive tokens, a quarter of a page.

  decode_spans  attention of one new token per request over its whole cache, or over listed spans of it
  span_keys     the mean latent of each listed span, kept beside the cache as its key
  span_scores   how much attention each span of a request gets, estimated from the span keys
  select_spans  the best spans of each request by their scores, and their token indices for the sparse decode
  read_kv       cached tokens read back as bf16 or fp32 latents

`listed()` gives the fixed cases, `draw()` more of the same ranges.  `prepare()` makes what a serving loop holds
before the call; `run()` makes one call, in plain torch operations or (with `own` set) through the library.
"""
import math

import torch

own = False

HEADS, DIM, NOPE, ROPE, GROUP = 64, 512, 448, 64, 64
PAGE, SPAN, PAGE_SPANS = 256, 64, 4
ROW_BYTES, PAGE_BYTES, SCALES_AT = 576, 149504, 147456
SCALE = DIM ** -0.5
WORKSPACE_BYTES = 48 << 20  # above what decode_spans and span_scores ask for here


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short chat turn, one request: latency
        dict(name="decode one request of 300", op="decode_spans", B=1, low=300, high=300, nsel=0),
        # a small batch of mixed prompts
        dict(name="decode 16 ragged", op="decode_spans", B=16, low=256, high=32768, nsel=0),
        # a full batch of long documents, every token attended: 2.45 GB of cache
        dict(name="decode 64 x 65536", op="decode_spans", B=64, low=65536, high=65536, nsel=0),
        # the same batch, 32 selected spans (2048 tokens) of each request
        dict(name="decode 64 x 32 spans", op="decode_spans", B=64, low=65536, high=65536, nsel=32),
        # after a decode step of 64 requests: the span each new token fell into
        dict(name="keys after a step", op="span_keys", B=64, low=1000, high=8192, new=1),
        # after prefill of 16 documents: every span of them
        dict(name="keys after prefill", op="span_keys", B=16, low=30001, high=65536, new=0),
        # spans of a small mixed batch
        dict(name="scores 16 ragged", op="span_scores", B=16, low=256, high=32768),
        # spans of a full batch of long documents
        dict(name="scores 64 x 65536", op="span_scores", B=64, low=65536, high=65536),
        # eight of one request's 128 spans: latency
        dict(name="select 8 of 128", op="select_spans", B=1, low=8192, high=8192, nsel=8, first=1, last=1),
        # a large batch of long ragged requests, 2048 tokens of each
        dict(name="select 32 of up to 2048", op="select_spans", B=256, low=1024, high=131072, nsel=32, first=1, last=2),
        # a prefix of one request read back for the next prompt chunk
        dict(name="read one prefix", op="read_kv", B=1, low=1337, high=1337, out="bf16"),
        # sixteen cached prefixes read back as fp32
        dict(name="read 16 prefixes", op="read_kv", B=16, low=2048, high=16384, out="fp32"),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["decode_spans", "decode_spans", "span_keys", "span_scores", "select_spans", "read_kv"])
    B = _log_uniform(rng, 1, 256 if op == "select_spans" else 64)
    top = {"decode_spans": 65536, "span_keys": 65536, "span_scores": 65536, "select_spans": 131072, "read_kv": 16384}[op]
    if op in ("read_kv", "span_keys"):
        B = min(B, 16)
    high = _log_uniform(rng, 1, top)
    low = high if rng.random() < 0.3 else _log_uniform(rng, 1, high)
    case = dict(op=op, B=B, low=low, high=high)
    if op == "decode_spans":
        case["nsel"] = rng.choice([0, _log_uniform(rng, 1, 64)])
    elif op == "span_keys":
        case["new"] = rng.choice([0, _log_uniform(rng, 1, 300)])
    elif op == "select_spans":
        case["nsel"] = _log_uniform(rng, 4, 64)
        case["first"], case["last"] = rng.choice([0, 1]), rng.choice([0, 1, 2])
    elif op == "read_kv":
        case["out"] = rng.choice(["bf16", "fp32"])
    return case


def _lens(case):
    """The requests' lengths: the same for every seed, so that a case has one amount of work."""
    low, high, B = case["low"], case["high"], case["B"]
    if low == high or B == 1:
        return [high] * B
    g = torch.Generator().manual_seed(7919 * B + 31 * low + high)
    return torch.randint(low, high + 1, (B,), generator=g).tolist()


def _spans(n):
    return -(-n // SPAN)


def work(case):
    lens, op = _lens(case), case["op"]
    B, spans = len(lens), [_spans(n) for n in lens]
    if op == "decode_spans":
        n = sum(lens) if not case["nsel"] else sum(min(case["nsel"] * SPAN, n) for n in lens)
        return dict(bytes=n * 584 + B * HEADS * (2 * DIM * 2 + 4) + B * case["nsel"] * 4, flops=n * HEADS * DIM * 4)
    if op == "span_keys":
        s = [min(_spans(n), _spans(n) - (n - min(case["new"], n)) // SPAN) if case["new"] else _spans(n) for n in lens]
        n = sum(k - (_spans(m) - c) * SPAN for k, m, c in zip(lens, lens, s))
        return dict(bytes=n * 584 + sum(s) * (DIM * 2 + 8), flops=n * DIM)
    if op == "span_scores":
        return dict(bytes=sum(spans) * (DIM * 2 + 4) + B * HEADS * DIM * 2, flops=sum(spans) * HEADS * DIM * 2)
    if op == "select_spans":
        return dict(bytes=sum(spans) * 4 + B * case["nsel"] * 4 * (1 + SPAN), flops=sum(spans))
    return dict(bytes=sum(lens) * (584 + 8 + DIM * (2 if case["out"] == "bf16" else 4)), flops=sum(lens) * NOPE)


# ---------------------------------------------------------------- what a serving loop holds
def _rows(cache):
    return cache.as_strided((cache.shape[0], PAGE, ROW_BYTES), (PAGE_BYTES, ROW_BYTES, 1))


def _scales(cache):
    return cache.as_strided((cache.shape[0], PAGE, 8), (PAGE_BYTES, 8, 1), SCALES_AT)


def _fill(cache, g):
    """Random latents in every page: N(0, 1), one row in a hundred 20 times larger, quantised as the cache holds them."""
    for at in range(0, cache.shape[0], 1024):
        rows, scales = _rows(cache[at:at + 1024]), _scales(cache[at:at + 1024])
        x = torch.randn((*rows.shape[:2], DIM), generator=g, device=cache.device)
        x *= 1.0 + 19.0 * (torch.rand(x.shape[:2], generator=g, device=cache.device) < 0.01).unsqueeze(-1)
        nope = x[..., :NOPE].unflatten(-1, (7, GROUP))
        mant, e = torch.frexp(nope.abs().amax(-1) / 448.0)
        e = torch.where(mant == 0.5, e - 1, e)
        rows[..., :NOPE] = torch.ldexp(nope, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
        rows[..., NOPE:] = x[..., NOPE:].to(torch.bfloat16).view(torch.uint8)
        scales[..., :7] = (e + 127).to(torch.uint8)
    return cache


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    lens, op = _lens(case), case["op"]
    B = len(lens)
    need = [-(-n // PAGE) for n in lens]
    pages, blocks = sum(need), max(need)
    s = dict(op=op, lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if op == "select_spans":
        # scores as span_scores gives them: the mass of a softmax over the spans, summed over 64 heads
        x = torch.randn((B, HEADS, blocks * PAGE_SPANS), generator=g, device=dev)
        dead = torch.arange(x.shape[-1], device=dev) >= torch.tensor([_spans(n) for n in lens], device=dev).view(B, 1, 1)
        s["scores"] = torch.softmax(x.masked_fill(dead, -math.inf), -1).sum(1)
        s.update(nsel=case["nsel"], first=case["first"], last=case["last"])
        return s
    table = torch.full((B, blocks), -1, dtype=torch.int32, device=dev)
    mapped = torch.arange(blocks, device=dev) < torch.tensor(need, device=dev).unsqueeze(1)
    table[mapped] = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    s["table"] = table
    if op in ("decode_spans", "span_scores"):
        s["q"] = torch.randn((B, HEADS, DIM), generator=g, device=dev).to(torch.bfloat16)
        s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    if op == "span_scores":
        # means of 64 tokens that differ from span to span
        s["keys"] = (torch.randn((pages, PAGE_SPANS, DIM), generator=g, device=dev) * 0.5).to(torch.bfloat16)
        return s
    s["cache"] = _fill(torch.zeros((pages, PAGE_BYTES), dtype=torch.uint8, device=dev), g)
    if op == "decode_spans":
        s["spans"] = None
        if case["nsel"]:
            # distinct spans in ascending order, -1 where a request has fewer
            r = torch.rand((B, blocks * PAGE_SPANS), generator=g, device=dev)
            nsp = torch.tensor([_spans(n) for n in lens], device=dev).unsqueeze(1)
            r[torch.arange(r.shape[1], device=dev) >= nsp] = 2.0
            width = min(case["nsel"], r.shape[1])
            at = torch.sort(torch.argsort(r, 1)[:, :width], 1).values
            at = torch.where(torch.gather(r, 1, at) < 2.0, at, -1)
            s["spans"] = torch.full((B, case["nsel"]), -1, dtype=torch.int32, device=dev)
            s["spans"][:, :width] = at
    elif op == "span_keys":
        req, span = [], []
        for b, n in enumerate(lens):
            at = range((n - min(case["new"], n)) // SPAN if case["new"] else 0, _spans(n))
            req += [b] * len(at)
            span += at
        s["req"] = torch.tensor(req, dtype=torch.int32, device=dev)
        s["span"] = torch.tensor(span, dtype=torch.int32, device=dev)
        s["keys"] = torch.zeros((pages, PAGE_SPANS, DIM), dtype=torch.bfloat16, device=dev)
    else:
        s["req"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(lens, device=dev)).to(torch.int32)
        s["pos"] = torch.cat([torch.arange(n, device=dev) for n in lens]).to(torch.int32)
        s["out"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    return s


# ---------------------------------------------------------------- plain forms
def _latents(rows, scales):
    """fp32 latents of raw rows [..., 576] and scale rows [..., 8]."""
    nope = rows[..., :NOPE].view(torch.float8_e4m3fn).float().unflatten(-1, (7, GROUP))
    nope = torch.ldexp(nope, scales[..., :7].int().unsqueeze(-1) - 127).flatten(-2)
    return torch.cat([nope, rows[..., NOPE:].view(torch.bfloat16).float()], -1)


def _attend(q, kv, valid):
    """q [B, H, D], kv [B, T, D], valid [B, T]: softmax(q kv^T) kv and the log-sum-exp; zeros and -inf without a token."""
    s = (q.float() @ kv.mT * SCALE).masked_fill(~valid.unsqueeze(1), -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ kv / total, 0.0)
    return out.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    cache, table, lens = s["cache"], s["table"].long(), s["lens"].long()
    if s["spans"] is None:
        page = table.clamp_min(0)
        kv = _latents(_rows(cache)[page], _scales(cache)[page]).flatten(1, 2)
        valid = torch.arange(kv.shape[1], device=kv.device) < lens.unsqueeze(1)
    else:
        span = s["spans"].long()
        pos = (span.unsqueeze(-1) * SPAN + torch.arange(SPAN, device=span.device)).flatten(1)
        valid = (span.repeat_interleave(SPAN, 1) >= 0) & (pos < lens.unsqueeze(1))
        pos = torch.where(valid, pos, 0)
        page = torch.gather(table, 1, pos // PAGE)
        kv = _latents(_rows(cache)[page, pos % PAGE], _scales(cache)[page, pos % PAGE])
    return _attend(s["q"], kv, valid)


def _plain_keys(s):
    cache, span, req = s["cache"], s["span"].long(), s["req"].long()
    page = s["table"].long()[req, span // PAGE_SPANS]
    slot = (span % PAGE_SPANS * SPAN).unsqueeze(1) + torch.arange(SPAN, device=span.device)
    x = _latents(_rows(cache)[page.unsqueeze(1), slot], _scales(cache)[page.unsqueeze(1), slot])
    n = (s["lens"].long()[req] - span * SPAN).clamp_max(SPAN)
    x = x * (torch.arange(SPAN, device=span.device) < n.unsqueeze(1)).unsqueeze(-1)
    s["keys"][page, span % PAGE_SPANS] = (x.sum(1) / n.unsqueeze(1)).to(torch.bfloat16)
    return s["keys"]


def _plain_scores(s):
    table, lens = s["table"].long(), s["lens"].long()
    keys = s["keys"].float()[table.clamp_min(0)].flatten(1, 2)
    dead = torch.arange(keys.shape[1], device=keys.device) * SPAN >= lens.unsqueeze(1)
    x = (s["q"].float() @ keys.mT * SCALE).masked_fill(dead.unsqueeze(1), -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return (p / p.sum(-1, keepdim=True)).sum(1)


def _plain_select(s):
    scores, lens, nsel = s["scores"], s["lens"].long().unsqueeze(1), s["nsel"]
    j = torch.arange(scores.shape[1], device=scores.device)
    count = (lens + SPAN - 1) // SPAN
    kept = (j < s["first"]) | (j >= count - s["last"])
    order = torch.where(j >= count, -math.inf, torch.where(kept, math.inf, scores.double()))
    width = min(nsel, scores.shape[1])
    at = torch.argsort(order, dim=1, descending=True, stable=True)[:, :width]
    at = torch.sort(torch.where(torch.gather(order, 1, at) > -math.inf, at, 1 << 30), 1).values
    spans = torch.full((scores.shape[0], nsel), -1, dtype=torch.int64, device=scores.device)
    spans[:, :width] = torch.where(at < 1 << 30, at, -1)
    pos = (spans.unsqueeze(-1) * SPAN + torch.arange(SPAN, device=spans.device)).flatten(1)
    pos = torch.where((pos >= 0) & (pos < lens), pos, -1)
    return spans.to(torch.int32), pos.to(torch.int32)


def _plain_read(s):
    req, pos = s["req"].long(), s["pos"].long()
    page = s["table"].long()[req, pos // PAGE]
    return _latents(_rows(s["cache"])[page, pos % PAGE], _scales(s["cache"])[page, pos % PAGE]).to(s["out"])


_PLAIN = dict(decode_spans=_plain_decode, span_keys=_plain_keys, span_scores=_plain_scores, select_spans=_plain_select,
              read_kv=_plain_read)


# ---------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if not own:
        return _PLAIN[op](s)
    import sparse_mla_decode_fp8_b200 as smla

    if op == "decode_spans":
        return smla.decode_spans(s["q"], s["cache"], s["table"], s["lens"], SCALE, spans=s["spans"], workspace=s["workspace"])
    if op == "span_keys":
        return smla.span_keys(s["cache"], s["table"], s["lens"], s["req"], s["span"], s["keys"])
    if op == "span_scores":
        return smla.span_scores(s["q"], s["keys"], s["table"], s["lens"], SCALE, workspace=s["workspace"])
    if op == "select_spans":
        return smla.select_spans(s["scores"], s["lens"], s["nsel"], keep_first=s["first"], keep_last=s["last"])
    return smla.read_kv(s["cache"], s["req"], s["pos"], s["table"], out_dtype=s["out"])


# ---------------------------------------------------------------- the definitions in 64 bits
def _byte_values(device):
    """The 256 e4m3 values by their bits: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = torch.arange(256, device=device)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.double() - 7))
    return torch.where(c >= 128, -v, v)


def _token_values(cache, code, values):
    """fp64 latents of tokens by code = page * 256 + slot."""
    flat = cache.view(-1)
    row = code // PAGE * PAGE_BYTES + code % PAGE * ROW_BYTES
    scale = code // PAGE * PAGE_BYTES + SCALES_AT + code % PAGE * 8
    col = torch.arange(NOPE, device=code.device)
    nope = values[flat[row.unsqueeze(1) + col].long()]
    nope = nope * 2.0 ** (flat[scale.unsqueeze(1) + col // GROUP].double() - 127)
    at = row.unsqueeze(1) + NOPE + 2 * torch.arange(ROPE, device=code.device)
    bits = (flat[at].int() | flat[at + 1].int() << 8) << 16
    return torch.cat([nope, bits.view(torch.float32).double()], 1)


def exact(case, seed):
    s, lens, op = prepare(case, seed), _lens(case), case["op"]
    if op == "select_spans":
        return None  # whole numbers
    table = s["table"].long()
    if op == "span_scores":
        got = torch.zeros((len(lens), table.shape[1] * PAGE_SPANS), dtype=torch.float64, device=table.device)
        for b, n in enumerate(lens):
            j = torch.arange(_spans(n), device=table.device)
            key = s["keys"][table[b, j // PAGE_SPANS], j % PAGE_SPANS].double()
            got[b, :len(j)] = torch.softmax(key @ s["q"][b].double().T * SCALE, 0).sum(1)
        return got
    values = _byte_values(table.device)

    def tokens(b, pos):
        return _token_values(s["cache"], table[b, pos // PAGE] * PAGE + pos % PAGE, values)

    if op == "decode_spans":
        outs, sums = [], []
        for b, n in enumerate(lens):
            if s["spans"] is None:
                pos = torch.arange(n, device=table.device)
            else:
                span = s["spans"][b][s["spans"][b] >= 0].long()
                pos = (span.unsqueeze(1) * SPAN + torch.arange(SPAN, device=table.device)).flatten()
                pos = pos[pos < n]
            kv = tokens(b, pos)
            x = s["q"][b].double() @ kv.T * SCALE
            sums.append(torch.logsumexp(x, 1))
            outs.append(torch.softmax(x, 1) @ kv)
        return torch.stack(outs), torch.stack(sums)
    if op == "span_keys":
        keys = torch.zeros(s["keys"].shape, dtype=torch.float64, device=table.device)
        for b, n in enumerate(lens):
            mine = s["span"][s["req"] == b].long()
            low = int(mine[0]) * SPAN
            pos = torch.arange(low, n, device=table.device)
            x = torch.zeros((len(mine) * SPAN, DIM), dtype=torch.float64, device=table.device)
            x[:n - low] = tokens(b, pos)
            count = (n - mine * SPAN).clamp_max(SPAN).unsqueeze(1)
            keys[table[b, mine // PAGE_SPANS], mine % PAGE_SPANS] = x.unflatten(0, (-1, SPAN)).sum(1) / count
        return keys
    return torch.cat([tokens(b, torch.arange(n, device=table.device)) for b, n in enumerate(lens)])
