"""Cases, plain forms and 64-bit values of the serving operators on a paged cache in 8 bits.

A row of the cache (one key or value of one key head) is held as e4m3 numbers c and one exponent
byte b, and stands for c * 2^(b - 127).  b is the smallest for which the row's largest magnitude is
at most 448 * 2^(b - 127); a row of zeros has b = 0.

  append   new keys and values are quantised into the pages of their sequences, keys (and the queries
           beside them) rotated by their position on the way;
  paged    attention of new queries over each sequence's pages;
  prefix   the same for a batch whose sequences begin with one long common prefix, whose pages are
           read once for all of them.

Tokens are packed one after another, as a projection leaves them: q [T][heads][d], k [T][kv_heads][d],
v [T][kv_heads][v]; sequence b owns tokens q_starts[b] .. q_starts[b + 1] - 1, the last tokens of its
seq_lens[b] cached ones.  Pages: k_pages [num_pages][kv_heads][page][d], k_scales [num_pages][kv_heads]
[page], the same of v; key j of sequence b is row j % page of page page_table[b][j / page].
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a small batch: 8 new tokens, latency alone counts.
        dict(name="append-decode-b8", op="append", dtype="bf16", B=8, heads=32, kv_heads=8, d=128,
             v=128, page=16, nq=1, ragged_q=False, len=2048, rot=128, interleaved=False),
        # Short odd prompts in fp32 with the irregular widths of the masked-attention workload
        # (d = 80, v = 96), adjacent-pair rotation of half the key's width.
        dict(name="append-prompts-f32-d80", op="append", dtype="f32", B=5, heads=8, kv_heads=8, d=80,
             v=96, page=32, nq=333, ragged_q=True, len=1000, rot=40, interleaved=True),
        # The prompts of 16 requests, about 40 thousand tokens in one call.
        dict(name="append-prompts-b16-n4096", op="append", dtype="bf16", B=16, heads=32, kv_heads=8,
             d=128, v=128, page=64, nq=4096, ragged_q=True, len=4096, rot=128, interleaved=False),
        # One user's decode step, a thousand tokens in: the smallest attention call.
        dict(name="paged-decode-b1-n1000", op="paged", dtype="bf16", B=1, heads=32, kv_heads=8, d=128,
             v=128, page=16, nq=1, ragged_q=False, len=1000, ragged_len=False, mask="causal",
             window=0),
        # The benchmark's decode step (8 sequences, 32 heads, 16384 keys, d = v = 128) from pages.
        dict(name="paged-decode-b8-n16384", op="paged", dtype="bf16", B=8, heads=32, kv_heads=32,
             d=128, v=128, page=64, nq=1, ragged_q=False, len=16384, ragged_len=False,
             mask="causal", window=0),
        # A busy server: 64 requests of very different lengths, 8 query heads to a key head.
        dict(name="paged-decode-b64-ragged", op="paged", dtype="bf16", B=64, heads=64, kv_heads=8,
             d=128, v=128, page=64, nq=1, ragged_q=False, len=32768, ragged_len=True,
             mask="causal", window=0),
        # Four guessed tokens of one very long document verified in one step.
        dict(name="paged-verify-n262147", op="paged", dtype="bf16", B=1, heads=32, kv_heads=8, d=128,
             v=128, page=32, nq=4, ragged_q=False, len=262147, ragged_len=False, mask="causal",
             window=0),
        # fp32 queries, irregular widths, a sliding window, odd lengths.
        dict(name="paged-window-f32-d80", op="paged", dtype="f32", B=7, heads=8, kv_heads=8, d=80,
             v=96, page=16, nq=2, ragged_q=True, len=4001, ragged_len=True, mask="window",
             window=1024),
        # A chunk of 512 prompt tokens for each of 4 requests, 8192 tokens into their prompts.
        dict(name="paged-chunk-nq512-n8192", op="paged", dtype="bf16", B=4, heads=32, kv_heads=8,
             d=128, v=128, page=64, nq=512, ragged_q=False, len=8192, ragged_len=False,
             mask="causal", window=0),
        # A few requests behind one instruction of 2000 tokens.
        dict(name="prefix-b8-n2000-d64", op="prefix", dtype="bf16", B=8, heads=16, kv_heads=16, d=64,
             v=64, page=16, nq=1, ragged_q=False, len=200, ragged_len=True, prefix=2000,
             mask="causal"),
        # Many samples of one long document: 64 sequences behind 16384 common tokens.
        dict(name="prefix-b64-n16384", op="prefix", dtype="bf16", B=64, heads=32, kv_heads=8, d=128,
             v=128, page=64, nq=1, ragged_q=False, len=512, ragged_len=True, prefix=16384,
             mask="causal"),
        # fp32 queries, irregular widths, two or fewer tokens each.
        dict(name="prefix-f32-b12-n3001", op="prefix", dtype="f32", B=12, heads=8, kv_heads=4, d=80,
             v=96, page=32, nq=2, ragged_q=True, len=77, ragged_len=True, prefix=3001,
             mask="causal"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "paged", "paged", "prefix"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    d = rng.choice((64, 128, 128, 80, 96, 112))
    v = rng.choice((d, d, d, 96, 64))
    kv = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice((1, 2, 3, 4, 7, 8))
    page = rng.choice((8, 16, 16, 32, 64, 128))
    B = _log(rng, 1, 64)
    case = dict(op=op, dtype=dtype, B=B, heads=kv * group, kv_heads=kv, d=d, v=v, page=page)
    if op == "append":
        nq = rng.choice((1, 1, 3, _log(rng, 5, 2048)))
        if dtype == "f32":
            nq = min(nq, 1024)
        case.update(nq=nq, ragged_q=rng.random() < 0.5, len=nq + _log(rng, 1, 1000),
                    rot=rng.choice((d, d, d // 2)), interleaved=rng.random() < 0.5)
        return case
    # At most 2^19 cached tokens of 8 key heads, or their like.
    most = max(64, (1 << 22) // (B * kv))
    n = _log(rng, 33, min(40000, most))
    nq = rng.choice((1, 1, 1, 2, 5, _log(rng, 8, 256)))
    nq = min(nq, n, max(1, 16384 // B))
    # At most 2^31 pairs of a query row and a key.
    while nq > 1 and B * nq * kv * group * n > (1 << 31):
        nq //= 2
    case.update(nq=nq, ragged_q=rng.random() < 0.4, len=n, ragged_len=rng.random() < 0.6)
    if op == "paged":
        mask = rng.choice(("causal", "causal", "none", "window"))
        case.update(mask=mask, window=_log(rng, 16, 8192) if mask == "window" else 0)
    else:
        n = max(nq, min(n, 600))
        p = _log(rng, 100, min(20000, max(200, (1 << 31) // (B * nq * kv * group))))
        case.update(len=n, prefix=p, mask=rng.choice(("causal", "causal", "none")))
    return case


def _spread(count, lo, hi, turn):
    """`count` whole numbers spread over lo .. hi, in no order."""
    return [lo + int((((b + 1) * 0.6180339887498949 + turn) % 1.0) * (hi - lo + 1)) for b in range(count)]


def _sizes(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    B = case["B"]
    nq = _spread(B, max(1, case["nq"] // 8), case["nq"], 0.3) if case["ragged_q"] else [case["nq"]] * B
    if case["op"] == "append":
        # A sequence of new tokens behind cached ones: none where the prompts fill the length.
        return nq, [max(a, n) for a, n in zip(nq, _spread(B, case["nq"], case["len"], 0.0))]
    if not case["ragged_len"]:
        return nq, [case["len"]] * B
    return nq, [max(a, n) for a, n in zip(nq, _spread(B, max(1, case["len"] // 16), case["len"], 0.0))]


# ---------------------------------------------------------------------------- inputs
def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x):
    """Rows x [.., width] as e4m3 numbers and exponent bytes [..]; each operation but the one
    rounding is exact."""
    top = x.abs().amax(-1)
    part, up = torch.frexp(top)  # top = part * 2^up, part in [1/2, 1); 448 = 7/8 * 2^9
    e = (up - 9 + (part > 0.875)).clamp(min=-126)
    z = x * _power(-e)[..., None].to(x.dtype)
    unit = _power(torch.frexp(z).exponent.clamp(min=-5) - 4).to(x.dtype)  # of three bits behind the first
    c = (torch.round(z / unit) * unit).float().to(torch.float8_e4m3fn)
    return c, torch.where(top > 0, e + 127, 0).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, dev, page = _TYPES[case["dtype"]], "cuda", case["page"]
    H, Hk, d, v = case["heads"], case["kv_heads"], case["d"], case["v"]
    nq, lens = _sizes(case)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    T, most = starts[-1], -(-max(lens) // page)
    needed = [-(-n // page) for n in lens]
    extra = -(-case["prefix"] // page) if case["op"] == "prefix" else 0
    num_pages = sum(needed) + extra + 3

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    # Keys have a few columns that are larger than the others, in each head the same.
    loud = 1 + 3 * (torch.rand(Hk, 1, d, generator=g, device=dev) < 1 / 16).float()
    k_pages, k_scales = _quantise(torch.randn(num_pages, Hk, page, d, generator=g, device=dev) * loud)
    v_pages, v_scales = _quantise(torch.randn(num_pages, Hk, page, v, generator=g, device=dev))
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(case["B"], most, dtype=torch.int32, device=dev)
    at = torch.tensor(needed, device=dev)
    cols = torch.arange(most, device=dev)
    used = cols[None, :] < at[:, None]
    table[used] = perm[: sum(needed)]
    s = dict(op=case["op"], q=rand(T, H, d), k_pages=k_pages, v_pages=v_pages, k_scales=k_scales,
             v_scales=v_scales, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             starts=torch.tensor(starts, dtype=torch.int32, device=dev) if case["ragged_q"] else None,
             B=case["B"], nq=max(nq))
    if case["op"] == "append":
        # k and v are columns of one projection's output, so their rows are not adjacent.
        kv = rand(T, Hk * (d + v))
        s.update(k=kv[:, : Hk * d].view(T, Hk, d), v=kv[:, Hk * d :].view(T, Hk, v),
                 interleaved=case["interleaved"],
                 inv_freq=torch.pow(10000.0, -torch.arange(0, case["rot"], 2, device=dev,
                                                            dtype=torch.float64) / case["rot"]).float())
    else:
        s.update(scale=1.0 / math.sqrt(d), mask=case["mask"], window=case.get("window", 0))
    if case["op"] == "prefix":
        s.update(prefix=case["prefix"], prefix_table=perm[sum(needed) : sum(needed) + extra].contiguous())
    return s


# ------------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def _own(s):
    import exact_tiled_softmax_gb300 as ex

    if "ws" not in s:  # made once, as a server does: outputs and workspace
        T, H = s["q"].shape[:2]
        s["y"] = torch.empty(T, H, s["v_pages"].shape[3], dtype=s["q"].dtype, device="cuda")
        s["L"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
        s["q_out"] = torch.empty_like(s["q"])
        shape = ex.paged_shape(s["q"], s["k_pages"], s["v_pages"], s["table"])
        size = ex.prefix_workspace_size if s["op"] == "prefix" else ex.paged_workspace_size
        s["ws"] = ex.workspace(size(shape), "cuda")
    if s["op"] == "append":
        ex.append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                        q_starts=s["starts"], q=s["q"], q_out=s["q_out"], inv_freq=s["inv_freq"],
                        interleaved=s["interleaved"], ws=s["ws"], k_scales=s["k_scales"],
                        v_scales=s["v_scales"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if s["op"] == "paged":
        return ex.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"],
                            s["mask"], s["window"], q_starts=s["starts"], y=s["y"], L=s["L"],
                            ws=s["ws"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    return ex.fwd_prefix(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix"],
                         s["table"], s["lens"], s["scale"], s["mask"], q_starts=s["starts"],
                         y=s["y"], L=s["L"], ws=s["ws"], k_scales=s["k_scales"],
                         v_scales=s["v_scales"])


def _tokens(s):
    """Of each token: its sequence, its number there, its position, counted from the cache's start."""
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    starts = s["starts"] if s["starts"] is not None else torch.arange(0, T + 1, T // s["B"], device="cuda")
    b = torch.searchsorted(starts[1:].long(), t, right=True)
    i = t - starts[b]
    return b, i, s["lens"][b] - (starts[b + 1] - starts[b]) + i


def _rotate(x, pos, inv_freq, interleaved):
    """In x's type, angles in 64 bits."""
    r = 2 * inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()
    c, n = angle.cos().to(x.dtype)[:, None], angle.sin().to(x.dtype)[:, None]
    y = x.clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., : r // 2], y[..., r // 2 : r])
    ra, rb = a * c - b * n, b * c + a * n
    a.copy_(ra)
    b.copy_(rb)
    return y


def _plain_append(s):
    b, _, pos = _tokens(s)
    page = s["k_pages"].shape[2]
    at, row = s["table"][b, pos // page].long(), pos % page
    # Keys in 64 bits: a value next to a border of its rounding keeps its side.
    k = _quantise(_rotate(s["k"].double(), pos, s["inv_freq"], s["interleaved"]))
    v = _quantise(s["v"].float())
    s["k_pages"].view(torch.uint8)[at, :, row] = k[0].view(torch.uint8)
    s["v_pages"].view(torch.uint8)[at, :, row] = v[0].view(torch.uint8)
    s["k_scales"][at, :, row] = k[1]
    s["v_scales"][at, :, row] = v[1]
    q = _rotate(s["q"].float(), pos, s["inv_freq"], s["interleaved"]).to(s["q"].dtype)
    return q, s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _gather(pages, scales, table):
    """[..][n pages] -> [..][kv_heads][keys][width], in 32 bits."""
    at = table.long()
    x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x = (x * _power(scales[at].long() - 127).float()[..., None]).transpose(-4, -3)
    return x.reshape(*x.shape[:-3], x.shape[-3] * x.shape[-2], x.shape[-1])


def _attend(q, k, v, allowed, scale):
    """Rows q [.., rows, d] over keys k [.., keys, d] where `allowed`; (Y, L)."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = torch.where(allowed, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    total = p.sum(-1, keepdim=True)
    y = (p @ v) / torch.where(total == 0, 1.0, total)
    return y, (m + total.log())[..., 0]


def _by_sequence(s):
    """The queries [B][kv_heads][nq * group][d] in 32 bits, and each one's token where it has one."""
    T, H, d = s["q"].shape
    Hk, nq = s["k_pages"].shape[1], s["nq"]
    b, i, pos = _tokens(s)
    q = torch.zeros(s["B"], nq, H, d, device="cuda")
    q[b, i] = s["q"].float()
    where = torch.full((s["B"], nq), -1, device="cuda", dtype=torch.long)
    where[b, i] = pos.long()
    q = q.view(s["B"], nq, Hk, H // Hk, d).transpose(1, 2).reshape(s["B"], Hk, nq * (H // Hk), d)
    return q, where, b, i


def _in_place(y, s, b, i):
    """[B][kv_heads][nq * group][width] -> [T][heads][width]."""
    B, Hk, rows = y.shape[:3]
    y = y.reshape(B, Hk, s["nq"], rows // s["nq"], -1).transpose(1, 2).reshape(B, s["nq"], -1, y.shape[3])
    return y[b, i]


def _keys_and_values(s, table):
    return _gather(s["k_pages"], s["k_scales"], table), _gather(s["v_pages"], s["v_scales"], table)


def _plain_paged(s):
    q, where, b, i = _by_sequence(s)
    k, v = _keys_and_values(s, s["table"])
    j = torch.arange(k.shape[2], device="cuda")
    ok = (j < s["lens"][:, None])[:, None, :].expand(-1, s["nq"], -1)
    if s["mask"] != "none":
        ok = ok & (j <= where[..., None])
    if s["mask"] == "window":
        ok = ok & (j > where[..., None] - s["window"])
    ok = ok.repeat_interleave(q.shape[2] // s["nq"], 1)[:, None]
    y, L = _attend(q, k, v, ok, s["scale"])
    return _in_place(y, s, b, i).to(s["q"].dtype), _in_place(L[..., None], s, b, i)[..., 0]


def _plain_prefix(s):
    q, where, b, i = _by_sequence(s)
    B, Hk, rows, d = q.shape
    # The prefix once for all rows, the rest for each sequence, then the two joined.
    k, v = (x[:, : s["prefix"]] for x in _keys_and_values(s, s["prefix_table"]))
    all_ = torch.ones(1, 1, 1, dtype=torch.bool, device="cuda")
    y0, L0 = _attend(q.transpose(0, 1).reshape(Hk, B * rows, d), k, v, all_, s["scale"])
    y0 = y0.view(Hk, B, rows, -1).transpose(0, 1)
    L0 = L0.view(Hk, B, rows).transpose(0, 1)
    k, v = _keys_and_values(s, s["table"])
    j = torch.arange(k.shape[2], device="cuda")
    ok = (j < s["lens"][:, None])[:, None, :].expand(-1, s["nq"], -1)
    if s["mask"] != "none":
        ok = ok & (j <= where[..., None])
    y1, L1 = _attend(q, k, v, ok.repeat_interleave(rows // s["nq"], 1)[:, None], s["scale"])
    L = torch.logaddexp(L0, L1)
    y = y0 * torch.exp(L0 - L)[..., None] + y1 * torch.exp(L1 - L)[..., None]
    return _in_place(y, s, b, i).to(s["q"].dtype), _in_place(L[..., None], s, b, i)[..., 0]


_PLAIN = {"append": _plain_append, "paged": _plain_paged, "prefix": _plain_prefix}


# ----------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, Hk, d, v = case["heads"], case["kv_heads"], case["d"], case["v"]
    nq, lens = _sizes(case)
    T = sum(nq)
    if case["op"] == "append":
        # Each token's q, k, v in, q out, k and v in 8 bits; six operations to a rotated pair, three to a
        # quantised element (magnitude and maximum, scaling, rounding).
        return {"bytes": T * (H * d * 2 * e + Hk * (d + v) * (e + 1) + 2 * Hk),
                "flops": 3 * T * ((H + Hk) * case["rot"] + Hk * (d + v))}
    rows = T * H * ((d + v) * e + 4)  # q in, Y and L out
    keys = pairs = 0
    for a, n in zip(nq, lens):
        first = 0
        if case["mask"] == "window":
            first = max(0, n - a + 1 - case["window"])
        keys += n - first
        for i in range(a):
            hi = n if case["mask"] == "none" else n - a + i + 1
            lo = max(0, hi - case["window"]) if case["mask"] == "window" else 0
            pairs += hi - lo
    if case["op"] == "prefix":
        keys += case["prefix"]
        pairs += T * case["prefix"]
    return {"bytes": rows + keys * Hk * (d + v + 2), "flops": 2 * pairs * H * (d + v)}


# ------------------------------------------------------------------ values in 64 bits
def _nearest(x):
    """Codes and exponent bytes of rows x [.., width] in 64 bits, from the list of all e4m3 numbers."""
    numbers = torch.arange(127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    border = (numbers[1:] + numbers[:-1]) / 2
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-126, 127)
    for _ in range(2):  # the logarithm may be off next to a whole number
        e = torch.where((top <= 448 * 2.0 ** (e - 1)) & (e > -126), e - 1, e)
        e = torch.where(top > 448 * 2.0 ** e, e + 1, e)
    z = (x / 2.0 ** e).abs()
    low, high = torch.bucketize(z, border), torch.bucketize(z, border, right=True)
    code = torch.where(low % 2 == 0, low, high)  # equal but on a border, where the even one counts
    return torch.copysign(numbers[code], x), torch.where(top > 0, e + 127, 0.0)[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    nq, lens = _sizes(case)
    page, H, Hk = case["page"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        q, kp, vp = s["q"].double(), s["k_pages"].double(), s["v_pages"].double()
        ke, ve = s["k_scales"].double(), s["v_scales"].double()
        k, t = s["k"].double(), 0
        half = case["rot"] // 2
        freq = s["inv_freq"].double()
        for b, (a, n) in enumerate(zip(nq, lens)):
            pos = torch.arange(n - a, n, device="cuda")
            turn = torch.polar(torch.ones(a, half, device="cuda", dtype=torch.float64),
                               torch.outer(pos.double(), freq))[:, None]
            for x in (q, k):
                part = x[t : t + a, :, : 2 * half]
                if case["interleaved"]:
                    z = torch.view_as_complex(part.reshape(a, -1, half, 2).contiguous()) * turn
                    part.copy_(torch.view_as_real(z).reshape(part.shape))
                else:
                    z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
                    part.copy_(torch.cat((z.real, z.imag), -1))
            at = s["table"][b].long()[torch.div(pos, page, rounding_mode="floor")]
            kp[at, :, pos % page], ke[at, :, pos % page] = _nearest(k[t : t + a])
            vp[at, :, pos % page], ve[at, :, pos % page] = _nearest(s["v"][t : t + a].double())
            t += a
        return q, kp, vp, ke.to(torch.uint8), ve.to(torch.uint8)
    ys, Ls, t = [], [], 0

    def rows(of, pages):
        x = s[of + "_pages"].view(torch.uint8).index_select(0, pages).view(torch.float8_e4m3fn).double()
        x = x * 2.0 ** (s[of + "_scales"].index_select(0, pages).double() - 127)[..., None]
        return x.transpose(0, 1).flatten(1, 2)

    for b, (a, n) in enumerate(zip(nq, lens)):
        pages = s["table"][b, : -(-n // page)].long()
        k, v = [rows("k", pages)[:, :n]], [rows("v", pages)[:, :n]]
        if case["op"] == "prefix":
            first = s["prefix_table"].long()
            for x, of in ((k, "k"), (v, "v")):
                x.insert(0, rows(of, first)[:, : case["prefix"]])
        k, v = torch.cat(k, 1), torch.cat(v, 1)
        before = case.get("prefix", 0)
        j = torch.arange(-before, n, device="cuda")
        pos = torch.arange(n - a, n, device="cuda")[:, None]
        ok = torch.ones(a, before + n, dtype=torch.bool, device="cuda")
        if case["mask"] != "none":
            ok &= j <= pos
        if case["mask"] == "window":
            ok &= j > pos - case["window"]
        out, stat = [], []
        for h in range(H):
            x = s["q"][t : t + a, h].double() @ k[h * Hk // H].T * s["scale"]
            x = x.masked_fill(~ok, float("-inf"))
            stat.append(torch.logsumexp(x, -1))
            out.append(torch.exp(x - stat[-1][:, None]) @ v[h * Hk // H])
        ys.append(torch.stack(out, 1))
        Ls.append(torch.stack(stat, 1))
        t += a
    return torch.cat(ys), torch.cat(Ls)
