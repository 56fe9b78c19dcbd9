"""Measured cases of the paged-serving operators: page assignment, rotary positions with the
cache write, and attention of several query tokens per row over the cache.

Each case is one call (or, for "cycle", the pair of calls) of a serving loop around the decode
step: the scheduler's request lengths become block tables and slots, the step's q/k/v rows get
their rotary positions and go to the cache, and the chunk's queries attend over it.  `run`
computes a pass in plain torch operations, or with `own` set through the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1000000.0  # rotary base of the cases


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of a full batch: every row adds a token, one in bs needs a page (latency)
        dict(name="pages-step-b256", op="pages", B=256, bs=16, ctx=16384, new=1, tail=0),
        # admission of a ragged prefill batch, 64 rows, up to 4096 new tokens each, bs 32
        dict(name="pages-prefill-b64", op="pages", B=64, bs=32, ctx=2000, new=4096, tail=37),
        # requests admitted with their prompts and released again: 500 rows of up to 2500 tokens
        dict(name="pages-cycle-b500", op="cycle", B=500, bs=16, ctx=0, new=2500, tail=0),
        # one decode step's rows of a Qwen3-0.6B-shaped layer, text positions (latency)
        dict(name="rotary-step-b64", op="rotary", N=64, Hq=16, Hkv=8, D=128, R=128, axes=1,
             inter=False, bs=32, paged=True, tail=0),
        # a ragged prefill of text and images, Qwen3-8B-shaped, three position axes, q/k/v cut
        # from one fused projection, a padded tail
        dict(name="rotary-prefill-3axes", op="rotary", N=16411, Hq=32, Hkv=8, D=128, R=128,
             axes=3, inter=False, bs=16, paged=True, tail=27),
        # partial rotary with interleaved pairs, small heads, contiguous cache, odd length
        dict(name="rotary-partial-d64", op="rotary", N=5001, Hq=16, Hkv=16, D=64, R=32, axes=2,
             inter=True, bs=16, paged=False, tail=0),
        # cross attention of one new token per row to encoder states of other lengths
        dict(name="cross-step-b32", op="attn", B=32, Hq=16, Hkv=16, D=64, bs=16, q_lo=1, q_hi=1,
             k_lo=200, k_hi=1500, causal=False, paged=True),
        # cross attention of ragged decoder prompts to ragged encoder states, contiguous cache
        dict(name="cross-ragged-b8", op="attn", B=8, Hq=16, Hkv=8, D=128, bs=16, q_lo=1,
             q_hi=700, k_lo=1, k_hi=4097, causal=False, paged=False),
        # a chunk of 512 tokens per row behind a 16K history (chunked prefill)
        dict(name="chunk-512-after-16k", op="attn", B=4, Hq=32, Hkv=8, D=128, bs=16, q_lo=512,
             q_hi=512, k_lo=16000, k_hi=16896, causal=True, paged=True),
        # a few drafted tokens verified against one long history: few rows, a long axis
        dict(name="verify-5-after-128k", op="attn", B=1, Hq=32, Hkv=8, D=128, bs=16, q_lo=5,
             q_hi=5, k_lo=131000, k_hi=131072, causal=True, paged=True),
        # whole prompts: four ragged prefills from an empty history
        dict(name="prefill-b4", op="attn", B=4, Hq=32, Hkv=8, D=128, bs=32, q_lo=1500,
             q_hi=4096, k_lo=0, k_hi=0, causal=True, paged=True),
        # the largest: 4096 decoder tokens against 16384 encoder states
        dict(name="cross-4096x16384", op="attn", B=1, Hq=32, Hkv=8, D=128, bs=64, q_lo=4096,
             q_hi=4096, k_lo=16384, k_hi=16384, causal=False, paged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["pages", "cycle", "rotary", "rotary", "attn", "attn", "attn"])
    bs = rng.choice([16, 32, 64])
    if op == "pages":
        new = rng.choice([1, _log_int(rng, 2, 4096)])
        B = _log_int(rng, 1, 1024 if new == 1 else max(2, 262144 // new))
        return dict(op=op, B=min(B, 1024), bs=bs, ctx=_log_int(rng, 1, 32768), new=new,
                    tail=rng.randint(0, 64))
    if op == "cycle":
        new = _log_int(rng, 1, 4096)
        return dict(op=op, B=min(1024, _log_int(rng, 1, max(2, 600000 // new))), bs=bs, ctx=0,
                    new=new, tail=rng.randint(0, 64))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    D = rng.choice([64, 128, 128])
    if op == "rotary":
        return dict(op=op, N=_log_int(rng, 1, 32768 * 10 // (Hkv * (G + 2))), Hq=Hkv * G, Hkv=Hkv,
                    D=D, R=rng.choice([D, D, D // 2]), axes=rng.choice([1, 2, 3]),
                    inter=rng.random() < 0.4, bs=bs, paged=rng.random() < 0.7,
                    tail=rng.randint(0, 30))
    B = _log_int(rng, 1, 32)
    q_hi = _log_int(rng, 1, max(1, 6000 // B))
    k_hi = _log_int(rng, 1, max(2, min(65536, int(1e9 / (B * q_hi * Hkv * G)))))
    causal = rng.random() < 0.5
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                k_lo=rng.randint(0 if causal else 1, k_hi), k_hi=k_hi, causal=causal,
                paged=rng.random() < 0.7)


def _lengths(case):
    """The rows' lengths of a case, a function of the case alone (so that work() knows them):
    [(held before, new)] of page cases, [(query tokens, cached tokens)] of attention cases."""
    def spread(i, n, lo, hi):  # odd steps over [lo, hi], not in order
        return lo if n <= 1 or hi <= lo else lo + (i * 7919 + 13) % n * (hi - lo) // (n - 1)
    B = case["B"]
    if case["op"] in ("pages", "cycle"):
        new = case["new"]
        return [(spread(i, B, (case["ctx"] + 1) // 2, case["ctx"]),
                 spread(i + 3, B, 1 if new == 1 else 0, new)) for i in range(B)]
    rows = []
    for i in range(B):
        nq = spread(i, B, case["q_lo"], case["q_hi"])
        nk = spread(i + 5, B, case["k_lo"], case["k_hi"])
        rows.append((nq, nk + nq if case["causal"] and case["k_hi"] == 0 else
                     max(nk, nq) if case["causal"] else nk))
    return rows


# ---------------------------------------------------------------------------
# inputs


class State:
    pass


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    s = State()
    s.case = dict(case)
    g = _gen(seed)
    if case["op"] in ("pages", "cycle"):
        _prepare_pages(s, case, g)
    elif case["op"] == "rotary":
        _prepare_rotary(s, case, g)
    else:
        _prepare_attn(s, case, g)
    return s


def _prepare_pages(s, case, g):
    rows, bs = _lengths(case), case["bs"]
    order = torch.randperm(len(rows), generator=g, device=DEV).tolist()
    rows = [rows[i] for i in order]
    ctx, new = [r[0] for r in rows], [r[1] for r in rows]
    mb = max(1, max(-(-(c + n) // bs) for c, n in rows))
    held = torch.tensor([-(-c // bs) for c in ctx], device=DEV)
    n_held = int(held.sum())
    pool = n_held + sum(-(-(c + n) // bs) - -(-c // bs) for c, n in rows) + 11
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    s.table = torch.full((len(rows), mb), -1, dtype=torch.int32, device=DEV)
    s.table[torch.arange(mb, device=DEV)[None, :] < held[:, None]] = perm[:n_held]
    s.free = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    s.free[:pool - n_held] = perm[n_held:]
    s.num_free = _i32([pool - n_held])
    s.ctx, s.new = _i32(ctx), _i32(new)
    s.bs, s.N = bs, max(1, sum(new)) + case["tail"]
    # what a serving loop allocates once
    s.num_free_out = torch.zeros_like(s.num_free)
    s.seq_lens = torch.zeros_like(s.ctx)
    s.cu = torch.zeros(len(rows) + 1, dtype=torch.int32, device=DEV)
    s.slots = torch.zeros(s.N, dtype=torch.int64, device=DEV)
    s.positions = torch.zeros(s.N, dtype=torch.int32, device=DEV)
    s.done = torch.ones(len(rows), dtype=torch.int32, device=DEV)
    s.ws = torch.zeros(256, dtype=torch.uint8, device=DEV)


def _axes(case):
    """Axis of each of the R/2 rotated pairs: sections of 1/4 time and the rest shared out, as
    images and video use them."""
    half, axes = case["R"] // 2, case["axes"]
    first = half if axes == 1 else half // 4
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (half - first)
            for i in range(half)]


def _inv_freq(case):
    return [THETA ** (-2.0 * i / case["R"]) for i in range(case["R"] // 2)]


def _prepare_rotary(s, case, g):
    N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
    total = N + case["tail"]
    s.qkv = _randn((total, (Hq + 2 * Hkv) * D), g)  # the fused projection's output
    s.q = s.qkv[:, :Hq * D].view(total, Hq, D)
    s.k = s.qkv[:, Hq * D:(Hq + Hkv) * D].view(total, Hkv, D)
    s.v = s.qkv[:, (Hq + Hkv) * D:].view(total, Hkv, D)
    # prompts of text with 24 x 32 image frames between, far into a long conversation
    base = int(torch.randint(0, 120000, (1,), generator=g, device=DEV))
    i = torch.arange(total, device=DEV)
    image = (i // 1024) % 2 == 1
    t = base + torch.where(image, i // 768, i)
    h = torch.where(image, base + i % 768 // 32, t)
    w = torch.where(image, base + i % 32, t)
    s.positions = torch.stack([t, h, w])[:case["axes"]].to(torch.int32).contiguous()
    if case["paged"]:
        bs = case["bs"]
        P = -(-total // bs) + 5
        page = torch.randperm(P, generator=g, device=DEV)
        s.slots = page[i // bs] * bs + i % bs
        s.K, s.V = (_randn((P, Hkv, bs, D), g) for _ in range(2))
    else:  # contiguous rows of T slots: slot b * T + t
        T = 1000
        rows = -(-total // T) + 1
        s.slots = (rows - 1 - i // T) * T + i % T
        s.K, s.V = (_randn((rows, Hkv, T, D), g) for _ in range(2))
    s.slots[N:] = -1  # padding behind the last token
    s.axis = torch.tensor(_axes(case), device=DEV)
    s.inv_freq = torch.tensor(_inv_freq(case), dtype=torch.float64, device=DEV)
    s.q_out = torch.zeros((total, Hq, D), dtype=torch.bfloat16, device=DEV)
    if own:
        import block_top_sparse_ksa_b200 as ksa
        s.rotary = ksa.Rotary(_inv_freq(case), _axes(case), interleaved=case["inter"])


def _prepare_attn(s, case, g):
    rows = _lengths(case)
    B, Hq, Hkv, D, bs = (case[k] for k in ("B", "Hq", "Hkv", "D", "bs"))
    nq, nk = [r[0] for r in rows], [r[1] for r in rows]
    N = sum(nq)
    s.cu = _i32([sum(nq[:i]) for i in range(B + 1)])
    s.seq_lens = _i32(nk)
    s.q = _randn((N, Hq, D), g)
    mb = max(1, max(-(-n // bs) for n in nk))
    if case["paged"]:
        held = torch.tensor([-(-n // bs) for n in nk], device=DEV)
        P = int(held.sum()) + 3
        page = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
        s.table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
        s.table[torch.arange(mb, device=DEV)[None, :] < held[:, None]] = page[:P - 3]
        s.K, s.V = (_randn((P, Hkv, bs, D), g) for _ in range(2))
    else:
        s.K, s.V = (_randn((B, Hkv, max(nk), D), g) for _ in range(2))
    s.max_q, s.max_k = max(nq), max(nk)
    s.out = torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=DEV)
    s.lse = torch.zeros((N, Hq), dtype=torch.float32, device=DEV)
    if own:
        import block_top_sparse_ksa_b200 as ksa
        s.ws = torch.zeros(ksa.ksa_chunk_attn_workspace(B, Hq, Hkv, D, mb * bs, N),
                           dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# one pass


def run(s):
    op = s.case["op"]
    if own:
        import block_top_sparse_ksa_b200 as ksa
        if op in ("pages", "cycle"):
            return _own_pages(ksa, s)
        return _own_rotary(ksa, s) if op == "rotary" else _own_attn(ksa, s)
    if op in ("pages", "cycle"):
        return _plain_pages(s)
    return _plain_rotary(s) if op == "rotary" else _plain_attn(s)


def _own_pages(ksa, s):
    ksa.ksa_assign_pages(s.ctx, s.new, s.table, s.free, s.num_free, s.bs, s.N,
                         num_free_out=s.num_free_out, seq_lens=s.seq_lens, cu_new=s.cu,
                         slots=s.slots, positions=s.positions, workspace=s.ws)
    if s.case["op"] == "cycle":
        ksa.ksa_release_pages(s.seq_lens, s.done, s.table, s.free, s.num_free_out, s.bs,
                              workspace=s.ws)
        return [s.table, s.free, s.num_free_out, s.seq_lens, s.cu, s.slots, s.positions]
    return [s.table, s.num_free_out, s.seq_lens, s.cu, s.slots, s.positions]


def _plain_pages(s):
    bs, N = s.bs, s.N
    ctx, new = s.ctx.long(), s.new.long()
    L = ctx + new
    held, blocks = (ctx + bs - 1) // bs, (L + bs - 1) // bs
    first = torch.cumsum(blocks - held, 0) - (blocks - held)  # pages taken by the rows before
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    F = s.num_free.long()
    j = torch.arange(s.table.shape[1], device=DEV)
    takes = (j >= held[:, None]) & (j < blocks[:, None])
    at = F - 1 - (first[:, None] + j - held[:, None])
    table = torch.where(takes, s.free[torch.where(takes, at, 0)], s.table)
    t = torch.arange(N, device=DEV)
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    real = t < cu[-1]
    pos = torch.where(real, ctx[row] + t - cu[row], -1)
    slots = torch.where(real, table[row, pos.clamp(min=0) // bs].long() * bs + pos % bs, -1)
    left = F - (blocks - held).sum()
    ints = [cu.to(torch.int32), slots, pos.to(torch.int32)]
    if s.case["op"] == "pages":
        return [table, left.to(torch.int32), L.to(torch.int32)] + ints
    # release: the stack takes the pages back, the last row's last page first
    back = blocks.sum()
    order = torch.cumsum(blocks, 0) - blocks
    gone = j < blocks[:, None]
    to = torch.where(gone, left + back - 1 - (order[:, None] + j), s.free.numel())
    free = torch.nn.functional.pad(s.free, (0, 1)).scatter(0, to.reshape(-1), table.reshape(-1))
    return [torch.where(gone, -1, table), free[:-1], (left + back).to(torch.int32),
            torch.zeros_like(s.seq_lens)] + ints


def _own_rotary(ksa, s):
    call = ksa.ksa_rotary_append_kv_paged if s.case["paged"] else ksa.ksa_rotary_append_kv
    call(s.q, s.k, s.v, s.positions, s.slots, s.K, s.V, s.rotary, q_out=s.q_out)
    return [s.q_out, s.K, s.V]


def _plain_rotary(s):
    case, R = s.case, s.case["R"]
    per = s.K.shape[2]
    angle = s.positions.double()[s.axis].T * s.inv_freq  # [N, R/2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float()
        if case["inter"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([y, x[..., R:]], -1).to(torch.bfloat16)

    real = s.slots >= 0
    page, off = s.slots[real] // per, s.slots[real] % per
    s.K[page, :, off] = turn(s.k)[real]
    s.V[page, :, off] = s.v[real]
    s.q_out[real] = turn(s.q)[real]
    return [s.q_out, s.K, s.V]


def _own_attn(ksa, s):
    mask = ksa.MASK_CAUSAL if s.case["causal"] else ksa.MASK_NONE
    if s.case["paged"]:
        ksa.ksa_chunk_attn_paged(s.q, s.K, s.V, s.table, s.cu, s.seq_lens, mask, out=s.out,
                                 lse=s.lse, workspace=s.ws)
    else:
        ksa.ksa_chunk_attn(s.q, s.K, s.V, s.cu, s.seq_lens, mask, out=s.out, lse=s.lse,
                           workspace=s.ws)
    return [s.out, s.lse]


def _plain_attn(s):
    c = s.case
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    K, V = s.K, s.V
    if c["paged"]:
        K, V = (x[s.table.clamp(min=0)].transpose(1, 2).reshape(B, Hkv, -1, D) for x in (K, V))
    K, V = K[:, :, :s.max_k].float(), V[:, :, :s.max_k].float()
    n = torch.arange(s.q.shape[0], device=DEV)
    row = torch.searchsorted(s.cu[1:], n.int(), right=True)
    at = n - s.cu[row]
    q = torch.zeros((B, s.max_q, Hq, D), dtype=torch.float32, device=DEV)
    q[row, at] = s.q.float()
    q = q.view(B, s.max_q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    z = (q @ K.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, -1, s.max_q, s.max_k)
    t = torch.arange(s.max_k, device=DEV)
    end = s.seq_lens[:, None]
    if c["causal"]:
        i = torch.arange(s.max_q, device=DEV)
        end = torch.minimum(end, end - (s.cu[1:] - s.cu[:-1])[:, None] + i + 1)
    seen = (t < end[..., None]).view(B, 1, 1, -1, s.max_k)
    z.masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    out = (z.view(B, Hkv, -1, s.max_k) @ V).view(*z.shape[:-1], D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, s.max_q, Hq, D)[row, at]
    lse = lse.permute(0, 3, 1, 2).reshape(B, s.max_q, Hq)[row, at]
    return [out.to(torch.bfloat16), lse]


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("pages", "cycle"):
        rows, bs = _lengths(case), case["bs"]
        tokens = sum(n for _, n in rows)
        taken = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in rows)
        # lengths in and out, pages off the stack and into the table, slots and positions
        moved = 12 * len(rows) + 8 * taken + 12 * (max(1, tokens) + case["tail"]) + 4 * len(rows)
        if op == "cycle":  # the pages off the table, onto the stack, and the table cleared
            moved += 12 * taken + 12 * len(rows)
        return {"bytes": moved, "flops": 4 * tokens}
    if op == "rotary":
        N, heads, D, R = case["N"], case["Hq"] + case["Hkv"], case["D"], case["R"]
        moved = 2 * 2 * N * (heads + case["Hkv"]) * D + N * (4 * case["axes"] + 8)
        return {"bytes": moved, "flops": 3 * N * heads * R + 40 * N * R // 2}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    pairs = keys = tokens = 0
    for n, L in _lengths(case):
        tokens += n
        keys += L
        pairs += n * L - n * (n - 1) // 2 if case["causal"] else n * L
    moved = tokens * Hq * (4 * D + 4) + keys * Hkv * 4 * D
    return {"bytes": moved, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# 64-bit values from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    return _exact_attn(s) if case["op"] == "attn" else None


def _exact_rotary(s):
    """Each pair as a complex number, times e^(i p f)."""
    case, R, N = s.case, s.case["R"], s.case["N"]
    p = torch.stack([s.positions[a, :N] for a in _axes(case)], 1).double()
    f = torch.tensor(_inv_freq(case), dtype=torch.float64, device=DEV)
    z = torch.polar(torch.ones_like(p), p * f)[:, None, :]

    def turned(x):
        y = x[:N].double().clone()
        lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["inter"] else (
            slice(0, R // 2), slice(R // 2, R))
        w = torch.complex(y[..., lo].clone(), y[..., hi].clone()) * z
        y[..., lo], y[..., hi] = w.real, w.imag
        return y

    q_out, K, V = s.q_out.double(), s.K.double(), s.V.double()
    q_out[:N] = turned(s.q)
    slot, per = s.slots[:N], s.K.shape[2]
    for h in range(case["Hkv"]):
        K[:, h].index_put_((slot // per, slot % per), turned(s.k)[:, h])
        V[:, h].index_put_((slot // per, slot % per), s.v[:N, h].double())
    return [q_out, K, V]


def _exact_attn(s):
    """Row by row and kv-head by kv-head, softmax by its definition."""
    c = s.case
    G, D = c["Hq"] // c["Hkv"], c["D"]
    pairs = sum(n * L for n, L in _lengths(c)) * c["Hq"]
    if pairs * D * 4 > 6e12:
        return None
    out = torch.zeros(s.q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s.q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    cu = s.cu.tolist()
    for b, L in enumerate(s.seq_lens.tolist()):
        n = cu[b + 1] - cu[b]
        if n == 0 or L == 0:
            continue
        for g in range(c["Hkv"]):
            if c["paged"]:
                pages = s.table[b, :-(-L // c["bs"])].long()
                k, v = (x[pages, g].reshape(-1, D)[:L].double() for x in (s.K, s.V))
            else:
                k, v = (x[b, g, :L].double() for x in (s.K, s.V))
            for h in range(g * G, (g + 1) * G):
                z = s.q[cu[b]:cu[b + 1], h].double() @ k.T / math.sqrt(D)
                if c["causal"]:
                    z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(L - n + 1),
                                      -math.inf)
                lse[cu[b]:cu[b + 1], h] = torch.logsumexp(z, -1)
                out[cu[b]:cu[b + 1], h] = torch.softmax(z, -1) @ v
    return [out, lse]
