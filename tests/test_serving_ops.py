"""Page assignment, rotary cache writes and chunk attention against plain 64-bit forms.

Whole numbers must be equal.  A bf16 value is off by at most half a step, 2^-8 of it, besides
the fp32 arithmetic before the rounding:
  rotary     sine and cosine within 1e-6 (fp32 turns and sincospi), products and sum 3 * 2^-24:
             2^-8 |x| + 2e-6 (|a| + |b|)
  attention  weights rounded to bf16 (2^-8 each), out rounded (2^-8), scores off by D 2^-24 of
             their terms' absolute sum (below 1e-4 here, so a weight by 2e-4):
             (2^-8 + 4e-4) sum w |v| + 2^-8 |out|;  lse 1e-4
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def ksa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import block_top_sparse_ksa_b200 as k
    k.lib()
    return k


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def randn(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# pages


def ref_assign(ctx, new, table, free, F, bs, N, T, num_pages):
    """The definition, row by row, with Python integers."""
    table, seq, slots, pos = table.copy(), [], [-1] * N, [-1] * N
    cu, at, asked, taken = [0], 0, 0, 0
    flags = 0
    for b, (c0, n0) in enumerate(zip(ctx, new)):
        c, n = min(max(c0, 0), T), min(max(n0, 0), T)
        bad = c != c0 or n != n0 or c + n > T or (n > 0 and at + n > N)
        held = -(-c // bs)
        need = 0 if bad else -(-(c + n) // bs) - held
        none = need > 0 and asked + need > F
        if bad:
            flags |= 1
        if none:
            flags |= 16
        if not bad and not none:
            for i in range(need):
                p = free[F - 1 - (asked + i)]
                if not 0 <= p < num_pages:
                    p = -1
                    flags |= 2
                table[b, held + i] = p
            taken += need
            for i in range(n):
                p = table[b, (c + i) // bs]
                pos[at + i] = c + i
                if 0 <= p < num_pages:
                    slots[at + i] = int(p) * bs + (c + i) % bs
                else:
                    flags |= 2
        seq.append(c if bad or none else c + n)
        asked += need
        at += n
        cu.append(min(at, N))
    return table, F - taken, seq, cu, slots, pos, flags


def page_state(rng, ctx, mb, bs, spare):
    """Tables of the held blocks and the stack of the other pages, in random order."""
    held = [min(mb, max(0, -(-c // bs))) for c in ctx]
    pool = sum(held) + spare
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(ctx), mb), -1, np.int32)
    k = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[k:k + h]
        k += h
    free = np.full(pool, -1, np.int32)
    free[:spare] = perm[k:]
    return table, free, spare, pool


def run_assign(ksa, ctx, new, table, free, F, bs, N, **kw):
    st = status()
    t, nf, out = torch.from_numpy(table).to(DEV), i32([F]), torch.full((1,), -7).to(DEV).int()
    seq, cu, slots, pos = ksa.ksa_assign_pages(i32(ctx), i32(new), t,
                                               torch.from_numpy(free).to(DEV), nf, bs, N,
                                               num_free_out=out, dev_status=st, **kw)
    assert int(nf) == F
    return t, out, seq, cu, slots, pos, int(st)


def same_assign(got, want):
    t, out, seq, cu, slots, pos, flags = got
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    assert int(out) == want[1]
    assert seq.tolist() == want[2] and cu.tolist() == want[3]
    assert slots.dtype == torch.int64 and slots.tolist() == want[4]
    assert pos.tolist() == want[5]
    assert flags == want[6]


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("B,new,tail", [(1, 1, 0), (1, 4000, 5), (7, 1, 0), (33, 100, 3),
                                        (1023, 2, 0), (1025, 1, 9), (2500, 3, 0), (300, 40, 1)])
def test_assign_pages(ksa, bs, B, new, tail):
    rng = np.random.default_rng(B * 100 + new + bs)
    mb = 4096 // bs + new // bs + 2
    ctx = rng.integers(0, 4096, B).tolist()
    ctx[0] = [0, bs, 2 * bs - 1][bs // 32]
    n = (rng.integers(0, new + 1, B) if new > 1 else np.ones(B, int)).tolist()
    need = sum(-(-(c + k) // bs) - -(-c // bs) for c, k in zip(ctx, n))
    table, free, F, pool = page_state(rng, ctx, mb, bs, need + 3)
    N = sum(n) + tail
    want = ref_assign(ctx, n, table, free, F, bs, N, mb * bs, pool)
    same_assign(run_assign(ksa, ctx, n, table, free, F, bs, N), want)


def test_assign_pages_refuses_whole_rows(ksa):
    """Out of pages, past the table, past the token axis, negative lengths: the row is refused
    whole and flagged, rows that need no page are still served."""
    bs, mb = 16, 8
    rng = np.random.default_rng(5)
    T = mb * bs
    cases = [
        ([0, 16, 3, 0, 5], [40, 16, 2, 1, 0], 4, 59),      # the stack runs out at row 3
        ([0, 16, 3, 0, 5], [40, 16, 2, 1, 0], 0, 59),      # an empty stack
        ([0, 120, 128, 129], [128, 9, 0, 1], 30, 200),     # L > T, c > T
        ([-1, 4, 4], [3, -2, 3], 10, 20),                  # negative lengths
        ([0, 0, 0], [10, 10, 10], 10, 25),                 # row 2 passes the token axis
        ([0, 0], [0, 0], 3, 0),                            # nothing new, no token axis
        ([0], [2 ** 31 - 1], 3, 7),
    ]
    for ctx, new, spare, N in cases:
        table, free, F, pool = page_state(rng, ctx, mb, bs, spare)
        if not pool:
            continue
        want = ref_assign(ctx, new, table, free, F, bs, N, T, pool)
        same_assign(run_assign(ksa, ctx, new, table, free, F, bs, N), want)


def test_assign_pages_skips_bad_page_ids(ksa):
    bs, mb = 16, 6
    table = np.full((2, mb), -1, np.int32)
    table[0, 0], table[1, 0] = 99, 1  # row 0's held block names no page
    free = np.array([0, 2, -5, 3, 77, 4], np.int32)
    ctx, new = [5, 16], [40, 33]
    want = ref_assign(ctx, new, table, free, 6, bs, 80, mb * bs, 6)
    got = run_assign(ksa, ctx, new, table, free, 6, bs, 80)
    same_assign(got, want)
    assert got[-1] == 2
    # a count outside the stack is clamped and flagged
    got = run_assign(ksa, [0], [16], table[:1], free, 9, bs, 16)
    assert got[-1] & 16 and got[0][0, 0] == 4 and int(got[1]) == 5


def test_assign_in_place_steps_in_a_graph(ksa):
    """The decode loop's form: lengths and count carried in place, captured once, replayed; 40
    steps over two pages per row, many CTAs."""
    B, bs, mb = 3000, 16, 6
    rng = np.random.default_rng(3)
    ctx0 = rng.integers(0, 40, B).astype(np.int32)
    table0, free0, F, pool = page_state(rng, ctx0.tolist(), mb, bs, 3 * B)
    lens, table = torch.from_numpy(ctx0).to(DEV), torch.from_numpy(table0).to(DEV)
    free, count = torch.from_numpy(free0).to(DEV), i32([F])
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    cu, slots, pos = (torch.zeros(k, dtype=d, device=DEV) for k, d in
                      ((B + 1, torch.int32), (B, torch.int64), (B, torch.int32)))

    def step():
        ksa.ksa_assign_pages(lens, one, table, free, count, bs, B, seq_lens=lens, cu_new=cu,
                             slots=slots, positions=pos, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(38):
        graph.replay()
    torch.cuda.synchronize()
    c, f, t = ctx0.tolist(), F, table0
    for _ in range(39):
        t, f, c, _, sl, ps, flags = ref_assign(c, [1] * B, t, free0, f, bs, B, mb * bs, pool)
        assert flags == 0
    assert lens.tolist() == c and int(count) == f
    np.testing.assert_array_equal(table.cpu().numpy(), t)
    assert slots.tolist() == sl and pos.tolist() == ps
    assert int(ws[:4].view(torch.int32)) == 0
    del graph


@pytest.mark.parametrize("B", [1, 5, 1024, 1025, 3000])
def test_release_undoes_assign(ksa, B):
    bs, mb = 16, 9
    rng = np.random.default_rng(B)
    new = rng.integers(0, mb * bs + 1, B).tolist()
    table, free, F, pool = page_state(rng, [0] * B, mb, bs, sum(-(-n // bs) for n in new) + 4)
    t, count = torch.from_numpy(table).to(DEV), i32([F])
    stack = torch.from_numpy(free).to(DEV)
    seq, *_ = ksa.ksa_assign_pages(i32([0] * B), i32(new), t, stack, count, bs, sum(new))
    assert int(count) == 4
    # some rows first, the others after; then nothing is left to give
    first = torch.from_numpy(rng.integers(0, 2, B).astype(np.int32)).to(DEV)
    t1 = t.clone()
    ksa.ksa_release_pages(seq, first, t, stack, count, bs)
    gone = [r for r in range(B) if first[r]]
    want = [int(p) for r in reversed(gone) for p in t1[r, :-(-new[r] // bs)].flip(0).tolist()]
    assert stack[4:int(count)].tolist() == want
    assert all((t[r] == -1).all() for r in gone) and all(seq[r] == 0 for r in gone)
    keep = [r for r in range(B) if not first[r]]
    assert torch.equal(t[keep], t1[keep])
    assert sorted(stack[:int(count)].tolist()) == sorted(set(stack[:int(count)].tolist()))
    ksa.ksa_release_pages(seq, torch.ones_like(first), t, stack, count, bs)
    assert int(count) == F and int(seq.abs().sum()) == 0 and bool((t == -1).all())
    assert sorted(stack[:F].tolist()) == sorted(free[:F].tolist())
    before = stack.clone()
    ksa.ksa_release_pages(seq, torch.ones_like(first), t, stack, count, bs)
    assert int(count) == F and torch.equal(stack, before)
    # all rows in one call: the stack as it was, bit for bit
    t, stack = torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV)
    seq, *_ = ksa.ksa_assign_pages(i32([0] * B), i32(new), t, stack, count, bs, sum(new))
    ksa.ksa_release_pages(seq, torch.ones_like(first), t, stack, count, bs)
    assert int(count) == F and torch.equal(stack.cpu(), torch.from_numpy(free))


def test_release_flags_bad_entries_and_a_full_stack(ksa):
    bs = 16
    table = torch.tensor([[1, 9], [2, 3]], dtype=torch.int32, device=DEV)
    stack, count, st = i32([0, -1, -1, -1]), i32([1]), status()
    seq = i32([20, 40])  # row 1's length is past its table
    ksa.ksa_release_pages(seq, i32([1, 1]), table, stack, count, bs, dev_status=st)
    # pushed: 3, 2, bad, (1 dropped: four places)
    assert stack.tolist() == [0, 3, 2, -1] and int(count) == 4
    assert int(st) == (1 | 2 | 16) and bool((table == -1).all()) and seq.tolist() == [0, 0]


def test_release_onto_the_largest_stack(ksa):
    """A full stack of 2^31 - 1 places: what does not fit is dropped, nothing is written before or
    behind the stack, and the count stays at its size."""
    bs, pages, room = 16, 2 ** 31 - 1, 3
    around = torch.full((pages + 64,), -7, dtype=torch.int32, device=DEV)
    stack = around[32:32 + pages]
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10)
    seq, count, st = i32([160, 155]), i32([pages - room]), status()
    ksa.ksa_release_pages(seq, i32([1, 1]), table, stack, count, bs, dev_status=st)
    assert int(st) == 16 and int(count) == pages and seq.tolist() == [0, 0]
    assert stack[-room:].tolist() == [19, 18, 17] and bool((table == -1).all())
    stack[-room:] = -7
    assert all(bool((part == -7).all()) for part in around.chunk(16))


# ---------------------------------------------------------------------------
# rotary


def ref_rotary(x, pos, axis, freq, inter):
    """x [N, H, D] bf16 -> rotated in fp64, and |a| + |b| of each element's pair."""
    P = len(freq)
    y, mag = x.double().cpu().numpy().copy(), np.abs(x.double().cpu().numpy())
    mag = mag.copy()
    ang = pos.cpu().numpy().astype(np.longdouble)[axis].T * np.asarray(freq, np.longdouble)
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    lo = slice(0, 2 * P, 2) if inter else slice(0, P)
    hi = slice(1, 2 * P, 2) if inter else slice(P, 2 * P)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mag[..., lo] = mag[..., hi] = np.abs(a) + np.abs(b)
    return y, mag


def close_rotary(got, want, mag, P):
    g = got.double().cpu().numpy()
    np.testing.assert_array_equal(g[..., 2 * P:], want[..., 2 * P:])  # behind the rotary dims
    assert (np.abs(g - want) <= HALF * np.abs(want) + 2e-6 * mag).all()


ROT = [  # N, Hq, Hkv, D, P, axes, interleaved, positions up to
    (1, 4, 2, 128, 64, 1, False, 10), (3, 1, 1, 64, 32, 3, True, 100),
    (70, 32, 8, 128, 64, 3, False, 1 << 20), (641, 5, 5, 64, 8, 2, True, 1 << 30),
    (1000, 7, 1, 128, 24, 2, False, 50000), (2300, 16, 8, 128, 64, 8, True, 3000),
    (593, 24, 8, 64, 16, 1, False, 2 ** 31 - 1), (592, 2, 1, 128, 56, 4, True, 1 << 24),
]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("N,Hq,Hkv,D,P,axes,inter,far", ROT)
def test_rotary_append(ksa, paged, N, Hq, Hkv, D, P, axes, inter, far):
    rng = np.random.default_rng(N + D + P)
    qkv = randn((N, (Hq + 2 * Hkv) * D + 8), N)  # columns of a wider projection
    q = qkv[:, :Hq * D].view(N, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(N, Hkv, D)
    pos = torch.from_numpy(rng.integers(-far, far, (axes, N)).astype(np.int32)).to(DEV)
    axis = [int(i) for i in rng.integers(0, axes, P)]
    freq = [10000.0 ** (-i / P) for i in range(P)]
    rot = ksa.Rotary(freq, axis, interleaved=inter, num_axes=axes)
    bs, T = 16, 100
    rows = -(-N // T) + 1
    K = randn((N // bs + 4, Hkv, bs, D) if paged else (rows, Hkv, T, D), 7)
    V = randn(tuple(K.shape), 8)
    per = K.shape[2]
    slots = rng.permutation(K.shape[0] * per)[:N].astype(np.int64)
    slots[::5] = -1
    if N > 2:
        slots[2] = K.shape[0] * per  # past the cache
    K0, V0 = K.clone(), V.clone()
    q_out = torch.full((N, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    st = status()
    call = ksa.ksa_rotary_append_kv_paged if paged else ksa.ksa_rotary_append_kv
    call(q, k, v, pos, torch.from_numpy(slots).to(DEV), K, V, rot, q_out=q_out, dev_status=st)
    assert int(st) == (2 if N > 2 else 0)
    real = (slots >= 0) & (slots < K.shape[0] * per)
    keep = torch.from_numpy(real).to(DEV)
    want, mag = ref_rotary(q, pos, axis, freq, inter)
    close_rotary(q_out[keep], want[real], mag[real], P)
    assert bool((q_out[~keep] == 3.0).all())
    pg = torch.from_numpy(slots[real] // per).to(DEV)
    off = torch.from_numpy(slots[real] % per).to(DEV)
    want, mag = ref_rotary(k, pos, axis, freq, inter)
    close_rotary(K[pg, :, off], want[real], mag[real], P)
    assert torch.equal(V[pg, :, off], v[keep])
    K0[pg, :, off], V0[pg, :, off] = K[pg, :, off], V[pg, :, off]
    assert torch.equal(K, K0) and torch.equal(V, V0)  # the rest of the cache is untouched


def test_rotary_parts(ksa):
    """In place, queries only, keys and values only, no rotation, default axis; one stream other
    than the current one."""
    N, Hq, Hkv, D = 37, 8, 2, 128
    q, k, v = randn((N, Hq, D), 1), randn((N, Hkv, D), 2), randn((N, Hkv, D), 3)
    pos = torch.arange(N, dtype=torch.int32, device=DEV) + 1000
    freq = [1e6 ** (-i / 64) for i in range(64)]
    rot = ksa.Rotary(np.array(freq))
    slots = torch.arange(N, device=DEV) + 5
    K, V = (torch.zeros((1, Hkv, 64, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = ksa.ksa_rotary_append_kv(q, k, v, pos, slots, K, V, rot)
    only = ksa.ksa_rotary_append_kv(q, None, None, pos, None, None, None, rot)
    assert torch.equal(only, out)
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    assert ksa.ksa_rotary_append_kv(None, k, v, pos, slots, K2, V2, rot) is None
    assert torch.equal(K2, K) and torch.equal(V2, V)
    q2 = q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ksa.ksa_rotary_append_kv(q2, None, None, pos[None], None, None, None, rot, q_out=q2,
                             stream=side)
    side.synchronize()
    assert torch.equal(q2, out)
    ksa.ksa_rotary_append_kv(None, k, v, None, slots, K2, V2, None)
    assert torch.equal(K2[0, :, 5:5 + N], k.transpose(0, 1)) and torch.equal(V2, V)
    empty = q[:0]
    assert ksa.ksa_rotary_append_kv(empty, None, None, pos[None, :0], None, None, None,
                                    rot).shape == (0, Hq, D)


@pytest.mark.parametrize("paged", [True, False])
def test_rotary_of_queries_with_slots_of_another_cache(ksa, paged):
    """Queries only: a slot says no more than whether the token is real, however far it is."""
    N, Hq, D = 9, 4, 64
    q, pos = randn((N, Hq, D), 4), torch.arange(N, dtype=torch.int32, device=DEV)
    rot, st = ksa.Rotary([0.3 ** i for i in range(32)]), status()
    want = ksa.ksa_rotary_append_kv(q, None, None, pos, None, None, None, rot)
    slots = torch.tensor([0, 5, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 62, -1, -2 ** 40],
                         device=DEV)
    out = torch.full_like(q, 3.0)
    call = ksa.ksa_rotary_append_kv_paged if paged else ksa.ksa_rotary_append_kv
    call(q, None, None, pos, slots, None, None, rot, q_out=out, dev_status=st)
    assert int(st) == 0
    assert torch.equal(out[:7], want[:7]) and bool((out[7:] == 3.0).all())


def test_rotary_offsets_past_32_bits(ksa):
    """A pool of more than 2^31 elements: the last page's rows land where they belong."""
    Hkv, bs, D = 8, 64, 128
    P = (2 ** 31) // (Hkv * bs * D) + 3
    K, V = (torch.empty((P, Hkv, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = randn((4, Hkv, D), 1), randn((4, Hkv, D), 2)
    slots = torch.tensor([P * bs - 1, 0, (P - 2) * bs + 7, P * bs], device=DEV)
    st = status()
    ksa.ksa_rotary_append_kv_paged(None, k, v, None, slots, K, V, None, dev_status=st)
    assert int(st) == 2
    assert torch.equal(K[P - 1, :, bs - 1], k[0]) and torch.equal(V[P - 1, :, bs - 1], v[0])
    assert torch.equal(K[0, :, 0], k[1]) and torch.equal(K[P - 2, :, 7], k[2])


@pytest.mark.parametrize("D", [128, 64])
def test_rotary_heads_past_32_bits(ksa, D):
    """A contiguous cache whose heads lie more than 2^31 elements apart: the last head's rows land
    in the last head, and no other row of the cache changes."""
    Hkv, T = 2, 2 ** 31 // D + 64
    K, V = (torch.zeros((1, Hkv, T, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = randn((4, Hkv, D), 1), randn((4, Hkv, D), 2)
    slots = torch.tensor([T - 1, 0, T // 2, -1], device=DEV)
    st = status()
    ksa.ksa_rotary_append_kv(None, k, v, None, slots, K, V, None, dev_status=st)
    assert int(st) == 0
    for x, src in ((K, k), (V, v)):
        for n, t in enumerate(slots.tolist()[:3]):
            assert torch.equal(x[0, :, t], src[n])
            x[0, :, t] = 0
        assert not any(bool(part.any()) for part in x.view(-1, D).chunk(16))


# ---------------------------------------------------------------------------
# chunk attention


def ref_attn(q, k, v, n, L, causal, scale):
    """One row in fp64: q [n, Hq, D], k and v [Hkv, L, D] -> out, lse, sum w |v|."""
    Hq, D = q.shape[1:]
    G = Hq // k.shape[0]
    k, v = k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
    z = torch.einsum("nhd,htd->hnt", q.double(), k) * scale
    if causal:
        i, t = torch.arange(n, device=DEV)[:, None], torch.arange(L, device=DEV)
        z = z.masked_fill(t > L - n + i, -torch.inf)
    lse = torch.logsumexp(z, -1) if L else torch.full((Hq, n), -torch.inf, device=DEV).double()
    w = torch.where(lse[..., None] == -torch.inf, 0.0, torch.exp(z - lse[..., None]))
    return ((w @ v).transpose(0, 1), lse.T, (w @ v.abs()).transpose(0, 1))


class Cache:
    """Random K/V of the given row lengths, contiguous or paged, everything a row does not hold
    poisoned with NaN and infinities."""

    def __init__(self, lens, Hkv, D, bs, paged, seed, T=None, mean=0.0):
        B = len(lens)
        self.lens, self.paged = lens, paged
        mb = max(1, -(-max(lens) // bs)) + 1
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.rows = [tuple((torch.randn((Hkv, L, D), generator=g, device=DEV) + mean)
                           .to(torch.bfloat16) for _ in range(2)) for L in lens]
        poison = [float("nan"), float("inf"), -float("inf")]
        if paged:
            need = sum(-(-L // bs) for L in lens)
            P = need + 2
            order = torch.randperm(P, generator=g, device=DEV).tolist()
            self.K, self.V = (torch.empty((P, Hkv, bs, D), dtype=torch.bfloat16, device=DEV)
                              for _ in range(2))
            for x in (self.K, self.V):
                for i, p in enumerate(poison):
                    x[i::3] = p
            table = np.full((B, mb), -1, np.int32)
            for b, L in enumerate(lens):
                for j in range(-(-L // bs)):
                    p = order.pop()
                    table[b, j] = p
                    part = slice(j * bs, min(L, (j + 1) * bs))
                    for x, src in zip((self.K, self.V), self.rows[b]):
                        x[p, :, :part.stop - part.start] = src[:, part]
            self.table = torch.from_numpy(table).to(DEV)
        else:
            T = T or max(1, max(lens)) + 3
            self.K, self.V = (torch.empty((B, Hkv, T, D), dtype=torch.bfloat16, device=DEV)
                              for _ in range(2))
            for x, w in ((self.K, 0), (self.V, 1)):
                for i, p in enumerate(poison):
                    x[:, :, i::3] = p
                for b, L in enumerate(lens):
                    x[b, :, :L] = self.rows[b][w]

    def call(self, ksa, q, cu, seq, mask, **kw):
        if self.paged:
            return ksa.ksa_chunk_attn_paged(q, self.K, self.V, self.table, cu, seq, mask, **kw)
        return ksa.ksa_chunk_attn(q, self.K, self.V, cu, seq, mask, **kw)


def check_attn(ksa, rows, Hq, Hkv, D, bs, paged, causal, seed, scale=0.0, mean=0.0, tail=0,
               **kw):
    """rows: (query tokens, cached tokens) of each row."""
    nq, lens = [r[0] for r in rows], [r[1] for r in rows]
    N = sum(nq) + tail
    q = randn((max(N, 1), Hq, D), seed + 1)[:N]
    cache = Cache(lens, Hkv, D, bs, paged, seed, mean=mean)
    cu = i32(np.concatenate([[0], np.cumsum(nq)]))
    out = torch.full((N, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((N, Hq), 5.0, device=DEV)
    st = status()
    cache.call(ksa, q, cu, i32(lens), ksa.MASK_CAUSAL if causal else ksa.MASK_NONE, scale=scale,
               out=out, lse=lse, dev_status=st, **kw)
    assert int(st) == 0
    at = 0
    for b, (n, L) in enumerate(rows):
        want, want_lse, mag = ref_attn(q[at:at + n], *cache.rows[b], n, L, causal,
                                       scale or D ** -0.5)
        got, got_lse = out[at:at + n].double(), lse[at:at + n].double()
        bound = (HALF + 4e-4) * mag + HALF * want.abs()
        off = ((got - want).abs() - bound).nan_to_num(nan=torch.inf)
        assert bool((off <= 1e-30).all()), (b, n, L, float(off.max()))
        empty = want_lse == -torch.inf
        assert bool((got_lse[empty] == -torch.inf).all()) and bool((got[empty] == 0).all())
        assert float((got_lse - want_lse)[~empty].abs().max().nan_to_num(nan=9.0)
                     if (~empty).any() else 0.0) <= 1e-4, (b, n, L)
        at += n
    assert bool((out[at:] == 5.0).all()) and bool((lse[at:] == 5.0).all())
    return cache, q, cu, out, lse


EDGES = [(1, 1), (0, 5), (1, 0), (3, 127), (2, 128), (5, 129), (33, 33), (1, 300), (64, 255),
         (31, 257), (7, 3), (0, 0), (130, 131), (1, 513), (260, 600)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv,bs,paged", [
    (128, 8, 2, 16, True), (128, 4, 4, 32, False), (64, 8, 1, 64, True), (64, 6, 2, 16, False),
    (128, 5, 1, 32, True), (128, 7, 1, 64, True), (64, 2, 2, 32, True), (128, 16, 2, 16, False),
    (64, 40, 2, 16, True), (128, 130, 2, 16, True), (64, 128, 1, 64, False)])
def test_chunk_attn_ragged(ksa, causal, D, Hq, Hkv, bs, paged):
    check_attn(ksa, EDGES, Hq, Hkv, D, bs, paged, causal, seed=D + Hq + bs, tail=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,Hq,Hkv,D,bs,paged", [
    ([(1, 20000)], 4, 1, 128, 16, True),             # one token, a long axis
    ([(5, 33001)], 32, 8, 128, 16, True),            # drafted tokens
    ([(1, 5000), (1, 17), (1, 0), (1, 9001)], 8, 8, 64, 32, True),
    ([(1, 4097)] * 32, 16, 8, 128, 16, False),       # a decode batch
    ([(700, 700)], 8, 2, 128, 64, True),             # a prompt
    ([(513, 5000), (1, 3000), (129, 129)], 4, 2, 64, 16, True),
    ([(2049, 2049)], 2, 1, 128, 16, False),
    ([(3, 70000)], 1, 1, 64, 64, False),
])
def test_chunk_attn_long(ksa, causal, rows, Hq, Hkv, D, bs, paged):
    check_attn(ksa, rows, Hq, Hkv, D, bs, paged, causal, seed=len(rows) + Hq)


@pytest.mark.parametrize("scale,mean", [(0.0, 1.0), (1.0, 0.0), (0.5, 2.0), (1e-3, 0.0)])
def test_chunk_attn_scales(ksa, scale, mean):
    """Peaked softmax (scale 1: weights of one token near 1) and flat ones; keys and values with
    a mean, so that the running maximum moves by much."""
    check_attn(ksa, [(40, 300), (200, 1000)], 4, 2, 64, 16, True, True, seed=3, scale=scale,
               mean=mean)


def test_chunk_attn_growing_scores(ksa):
    """Scores that rise with every key tile by far more than a rescaling threshold, then fall."""
    D, L, n = 64, 1500, 70
    cache = Cache([L], 1, D, 16, False, 9)
    ramp = torch.cat([torch.linspace(-6, 6, L // 2), torch.linspace(6, -6, L - L // 2)]).to(DEV)
    k = cache.rows[0][0]
    k[:] = ramp[None, :, None].to(torch.bfloat16)
    cache.K[0, :, :L] = k
    q = torch.ones((n, 2, D), dtype=torch.bfloat16, device=DEV)
    cu, seq = i32([0, n]), i32([L])
    lse = torch.empty((n, 2), device=DEV)
    out, _ = cache.call(ksa, q, cu, seq, ksa.MASK_NONE, lse=lse)
    want, want_lse, mag = ref_attn(q, k, cache.rows[0][1], n, L, False, D ** -0.5)
    assert bool(((out.double() - want).abs() <= (HALF + 4e-4) * mag + HALF * want.abs()).all())
    assert float((lse.double() - want_lse).abs().max()) <= 1e-4


def test_chunk_attn_strided_q_streams_and_no_lse(ksa):
    """q as columns of a projection, lse not asked for, a caller's workspace used by calls one
    after another on another stream, results equal bit for bit."""
    rows = [(9, 2000), (65, 700)]
    cache, q, cu, out, lse = check_attn(ksa, rows, 4, 2, 128, 16, True, True, seed=21)
    N = q.shape[0]
    wide = torch.zeros((N, 4 * 128 + 256), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:64 + 512] = q.reshape(N, -1)
    qs = wide[:, 64:64 + 512].view(N, 4, 128)
    ws = torch.zeros(ksa.ksa_chunk_attn_workspace(2, 4, 2, 128, cache.table.shape[1] * 16, N),
                     dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got, none = cache.call(ksa, qs, cu, i32([2000, 700]), ksa.MASK_CAUSAL, workspace=ws,
                               stream=side)
        side.synchronize()
        assert none is None and torch.equal(got, out)


def test_chunk_attn_bad_device_data(ksa):
    """Lengths outside the cache are clamped, offsets outside the tokens too, page ids outside the
    pool are left out; each sets its flag and nothing faults."""
    Hq, Hkv, D, bs = 4, 2, 64, 16
    cache = Cache([100, 40], Hkv, D, bs, True, 4)
    q = randn((30, Hq, D), 1)
    cache.table[0, 2] = 10 ** 6
    cache.table[0, 4] = -3
    st = status()
    out, _ = cache.call(ksa, q, i32([0, 20, 30]), i32([100, 40]), ksa.MASK_NONE, dev_status=st)
    assert int(st) == 2
    k, v = (torch.cat([x[:, :32], x[:, 48:64], x[:, 80:]], 1) for x in cache.rows[0])
    want, _, mag = ref_attn(q[:20], k, v, 20, k.shape[1], False, D ** -0.5)
    assert bool(((out[:20].double() - want).abs() <= (HALF + 4e-4) * mag + HALF * want.abs()).all())
    cache = Cache([64, 64], Hkv, D, bs, False, 4, T=64)
    full, _ = cache.call(ksa, q, i32([0, 20, 30]), i32([64, 64]), ksa.MASK_NONE)
    for lens, cu in (([65, 2 ** 31 - 1], [0, 20, 30]), ([64, 64], [0, 20, 31]),
                     ([64, 64], [-1, 20, 2 ** 31 - 1])):
        st = status()
        out, _ = cache.call(ksa, q, i32(cu), i32(lens), ksa.MASK_NONE, dev_status=st)
        assert int(st) == 1 and torch.equal(out, full)
    st = status()
    out, _ = cache.call(ksa, q, i32([0, 20, 30]), i32([-5, 64]), ksa.MASK_NONE, dev_status=st)
    assert int(st) == 1 and bool((out[:20] == 0).all()) and torch.equal(out[20:], full[20:])
    st = status()
    out = torch.full_like(q, 2.0)  # descending offsets: bounded, flagged, no token past N
    cache.call(ksa, q, i32([0, 30, 10]), i32([64, 64]), ksa.MASK_NONE, out=out, dev_status=st)
    assert int(st) == 1


def test_chunk_attn_offsets_past_32_bits(ksa):
    """Rows at the end of pools of more than 2^31 elements, paged and contiguous."""
    Hkv, bs, D, L, n = 2, 64, 128, 200, 6
    src = [randn((Hkv, 256, D), s) for s in (1, 2)]
    q = randn((n, 4, D), 3)
    want, _, mag = ref_attn(q, src[0][:, :L], src[1][:, :L], n, L, True, D ** -0.5)
    P = 2 ** 31 // (Hkv * bs * D) + 9
    K, V = (torch.empty((P, Hkv, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ids = [P - 1, 0, P - 3, P - 2]
    for x, s in zip((K, V), src):
        for j, p in enumerate(ids):
            x[p] = s[:, j * bs:(j + 1) * bs]
    got, _ = ksa.ksa_chunk_attn_paged(q, K, V, i32([ids]), i32([0, n]), i32([L]))
    assert bool(((got.double() - want).abs() <= (HALF + 4e-4) * mag + HALF * want.abs()).all())
    del K, V
    T = 2 ** 30 // (Hkv * D) + 256
    K, V = (torch.empty((3, Hkv, T, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for x, s in zip((K, V), src):
        x[2, :, :256] = s
    got, _ = ksa.ksa_chunk_attn(q, K, V, i32([0, 0, 0, n]), i32([0, 0, L]))
    assert bool(((got.double() - want).abs() <= (HALF + 4e-4) * mag + HALF * want.abs()).all())


def test_chunk_attn_single_tokens_agree_with_decode_attention(ksa):
    """One query token per row: the dense decode attention's result."""
    lens = [700, 16, 1, 2050]
    cache = Cache(lens, 4, 128, 16, True, 6)
    q = randn((4, 16, 128), 2)
    lse = torch.empty((4, 16), device=DEV)
    out, _ = cache.call(ksa, q, i32(range(5)), i32(lens), ksa.MASK_CAUSAL, lse=lse)
    lse2 = torch.empty((4, 16), device=DEV)
    want, _ = ksa.ksa_sparse_decode_attn_paged(q, cache.K, cache.V, cache.table, i32(lens),
                                               lse=lse2)
    for b, L in enumerate(lens):
        _, _, mag = ref_attn(q[b:b + 1], *cache.rows[b], 1, L, True, 128 ** -0.5)
        off = (out[b:b + 1].double() - want[b:b + 1].double()).abs()
        assert bool((off <= 2 * (HALF + 4e-4) * mag + HALF * want[b:b + 1].abs()).all())
    assert float((lse - lse2).abs().max()) <= 2e-4


# ---------------------------------------------------------------------------
# the operators as a serving loop uses them


def test_serving_steps_end_to_end(ksa):
    """Two prefill chunks and decode steps of a ragged batch: lengths -> pages and slots ->
    rotary and cache write -> chunk attention, then summaries and the block-sparse decode step
    (every block kept) on the same pages, every output against dense fp64 attention; then the
    rows are released and their pages serve the next requests."""
    Hq, Hkv, D, bs, B, mb = 8, 2, 128, 16, 3, 24
    P = 40
    rng = np.random.default_rng(1)
    K, V = (torch.full((P, Hkv, bs, D), float("nan"), dtype=torch.bfloat16, device=DEV)
            for _ in range(2))
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    free = torch.from_numpy(rng.permutation(P).astype(np.int32)).to(DEV)
    count, lens = i32([P]), torch.zeros(B, dtype=torch.int32, device=DEV)
    freq = [1e6 ** (-i / 64) for i in range(64)]
    axis = [i * 3 // 64 for i in range(64)]
    rot, st = ksa.Rotary(freq, axis), status()
    hist = [[], [], []]  # each row's (rotated k, v) so far, fp64 of the bf16 in the cache

    def step(new, seed):
        N = sum(new)
        _, cu, slots, pos = ksa.ksa_assign_pages(lens, i32(new), table, free, count, bs, N + 2,
                                                 seq_lens=lens, dev_status=st)
        qkv = randn((N + 2, (Hq + 2 * Hkv) * D), seed)
        q = qkv[:, :Hq * D].view(-1, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(-1, Hkv, D)
        v = qkv[:, (Hq + Hkv) * D:].view(-1, Hkv, D)
        p3 = torch.stack([pos, pos // 2, pos % 7])
        qr = ksa.ksa_rotary_append_kv_paged(q, k, v, p3, slots, K, V, rot, dev_status=st)
        c = cu.tolist()
        assert c[-1] == N and slots[N:].tolist() == [-1, -1]
        wk, mk = ref_rotary(k, p3, axis, freq, False)
        for b in range(B):
            for t in range(c[b], c[b + 1]):
                s = int(slots[t])
                row = K[s // bs, :, s % bs]
                close_rotary(row[None], wk[t:t + 1], mk[t:t + 1], 64)
                hist[b].append((row.clone(), v[t]))
        return qr, cu, c

    def check(out, qr, c, slack=0.0):
        for b in range(B):
            n = c[b + 1] - c[b]
            if not n:
                continue
            k, v = (torch.stack([h[w] for h in hist[b]], 1) for w in (0, 1))
            want, _, mag = ref_attn(qr[c[b]:c[b + 1]], k, v, n, len(hist[b]), True, D ** -0.5)
            off = (out[c[b]:c[b + 1]].double() - want).abs()
            assert bool((off <= (HALF + 4e-4) * mag + HALF * want.abs() + slack).all())

    for new, seed in (([130, 1, 40], 1), ([5, 20, 0], 2)):
        qr, cu, c = step(new, seed)
        out, _ = ksa.ksa_chunk_attn_paged(qr, K, V, table, cu, lens, ksa.MASK_CAUSAL,
                                          dev_status=st)
        check(out, qr, c)
    S = ksa.ksa_build_block_summaries_paged(K, table, lens, dev_status=st)
    for seed in range(3, 6):
        qr, cu, c = step([1, 1, 1], seed)
        idx, cnt = ksa.ksa_decode_select_blocks_paged(qr[:B].contiguous(), K, table, S, lens, mb,
                                                      dev_status=st)
        out, _ = ksa.ksa_sparse_decode_attn_paged(qr[:B].contiguous(), K, V, table, lens, idx,
                                                  cnt, tokens_per_idx=bs, dev_status=st)
        check(out, qr, c)
    assert int(st) == 0 and lens.tolist() == [138, 24, 43]
    assert int(count) == P - (9 + 2 + 3)
    ksa.ksa_release_pages(lens, i32([1, 0, 1]), table, free, count, bs, dev_status=st)
    hist[0], hist[2] = [], []
    qr, cu, c = step([33, 2, 1], 9)
    out, _ = ksa.ksa_chunk_attn_paged(qr, K, V, table, cu, lens, ksa.MASK_CAUSAL, dev_status=st)
    check(out, qr, c)
    assert int(st) == 0 and int(count) == P - (3 + 2 + 1)


def test_chunk_attn_captured_in_two_graphs(ksa):
    """Two graphs on one workspace, replayed in turn: each gives the eager result."""
    rows = [(3, 9000), (17, 400)]
    cache, q, cu, out, lse = check_attn(ksa, rows, 8, 2, 128, 16, True, True, seed=31)
    seq = i32([9000, 400])
    ws = torch.zeros(ksa.ksa_chunk_attn_workspace(2, 8, 2, 128, cache.table.shape[1] * 16, 20),
                     dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(out) for _ in range(2)]
    masks = (ksa.MASK_CAUSAL, ksa.MASK_NONE)
    eager = [cache.call(ksa, q, cu, seq, m, workspace=ws)[0] for m in masks]
    torch.cuda.synchronize()
    graphs = []
    for m, o in zip(masks, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            cache.call(ksa, q, cu, seq, m, out=o, workspace=ws)
    for _ in range(3):
        for gr, o, want in zip(graphs, outs, eager):
            o.fill_(-7.0)
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)
    assert torch.equal(eager[0], out)
    del graphs


def test_serving_calls_refuse_wrong_tensors(ksa):
    """Type, shape, layout and device of every tensor, by name, before anything is launched."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    q, K, cu, seq = bf(4, 4, 64), bf(2, 2, 32, 64), i32([0, 3, 4]), i32([5, 6])
    ok = lambda **kw: ksa.ksa_chunk_attn(**{**dict(q=q, K=K, V=K, cu_q=cu, seq_lens=seq), **kw})
    ok()
    for kw, kind in ((dict(q=q.float()), TypeError), (dict(K=K.half()), TypeError),
                     (dict(V=K[:, :, :16]), ValueError), (dict(K=K.transpose(2, 3)), ValueError),
                     (dict(cu_q=cu[:2]), ValueError), (dict(cu_q=cu.long()), TypeError),
                     (dict(seq_lens=seq.cpu()), TypeError), (dict(out=bf(4, 4, 32)), ValueError),
                     (dict(out=q.float()), TypeError), (dict(lse=bf(4, 4)), TypeError),
                     (dict(lse=torch.zeros((4, 3), device=DEV)), ValueError),
                     (dict(q=q.transpose(0, 1)), ValueError),
                     (dict(workspace=torch.zeros(9, dtype=torch.uint8)), TypeError),
                     (dict(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)),
                      ksa.KsaError)):
        with pytest.raises(kind):
            ok(**kw)
    table, free, one = i32([[0, 1]]), i32([0, 1, 2]), i32([1])
    ok = lambda **kw: ksa.ksa_assign_pages(**{**dict(
        ctx_lens=one, new_lens=one, block_table=table, free_pages=free, num_free=one,
        block_size=16, num_tokens=2), **kw})
    for kw, kind in ((dict(ctx_lens=i32([1, 2])), ValueError),
                     (dict(new_lens=one.long()), TypeError),
                     (dict(block_table=table.T), ValueError), (dict(num_free=one.cpu()), TypeError),
                     (dict(slots=i32([0, 0])), TypeError), (dict(block_size=8), ksa.KsaError),
                     (dict(positions=i32([0])), ValueError), (dict(num_tokens=-1, slots=one.long(),
                                                                   positions=one), ValueError)):
        with pytest.raises(kind):
            ok(**kw)
    rot, k = ksa.Rotary([0.5] * 32), bf(4, 2, 64)
    slots, pos = torch.arange(4, device=DEV), i32([0, 1, 2, 3])
    ok = lambda **kw: ksa.ksa_rotary_append_kv(**{**dict(
        q=q, k=k, v=k, positions=pos, slots=slots, K=K, V=K.clone(), rotary=rot), **kw})
    ok()
    for kw, kind in ((dict(k=bf(3, 2, 64)), ValueError), (dict(v=k.float()), TypeError),
                     (dict(slots=slots.int()), TypeError), (dict(positions=pos[:3]), ValueError),
                     (dict(positions=pos.cpu()), TypeError), (dict(positions=None), TypeError),
                     (dict(slots=None), ValueError), (dict(q_out=bf(4, 4, 32)), ValueError),
                     (dict(rotary=ksa.Rotary([0.5] * 32, num_axes=2)), ValueError),
                     (dict(rotary=ksa.Rotary([0.5] * 40)), ksa.KsaError),
                     (dict(V=K[:1]), ValueError), (dict(K=bf(2, 2, 64)), ValueError)):
        with pytest.raises(kind):
            ok(**kw)


def test_chunk_attn_non_finite_scores(ksa):
    """A NaN or infinite key reaches exactly the queries that see it; one behind a causal query
    does not, and huge finite scores stay finite.  Whole and split items."""
    n, L, D = 6, 700, 64
    for bad in (float("nan"), float("inf"), -float("inf")):
        for L in (700, 9000):
            cache = Cache([L, 300], 1, D, 16, False, 12)
            q = randn((n + 3, 2, D), 5).abs() + 0.5  # no score of an infinite key is a NaN sum
            cache.K[0, 0, L - 3] = bad  # seen by the last three of the six queries
            out, lse = (torch.empty((n + 3, 2, D), dtype=torch.bfloat16, device=DEV),
                        torch.empty((n + 3, 2), device=DEV))
            cache.call(ksa, q, i32([0, n, n + 3]), i32([L, 300]), ksa.MASK_CAUSAL, out=out,
                       lse=lse)
            k = cache.K[0, :, :L]
            want, want_lse, mag = ref_attn(q[:n], k, cache.rows[0][1], n, L, True, D ** -0.5)
            seen = torch.arange(n, device=DEV) >= n - 3
            if bad == -float("inf"):  # weighs nothing
                assert bool(torch.isfinite(out.float()).all())
                seen[:] = False
            else:
                assert bool(out[:n][seen].isnan().all()) and bool(lse[:n][seen].isnan().all())
            off = (out[:n].double() - want).abs() - (HALF + 4e-4) * mag - HALF * want.abs()
            assert bool((off[~seen] <= 0).all())
            assert float((lse[:n].double() - want_lse)[~seen].abs().max()) <= 1e-4
            assert bool(torch.isfinite(out[n:].float()).all())
    # scores up to 64 * 200 * 200 / 8: one weight is 1, nothing overflows
    cache = Cache([400], 1, D, 16, True, 13)
    q = randn((40, 4, D), 6) * 200
    cache.K *= 200
    lse = torch.empty((40, 4), device=DEV)
    out, _ = cache.call(ksa, q, i32([0, 40]), i32([400]), ksa.MASK_CAUSAL, lse=lse)
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())


def test_chunk_attn_many_rows_and_heads(ksa):
    """More rows than one look-up takes, in mixed depths, some empty; items cut by the mean row."""
    rng = np.random.default_rng(2)
    for B, far in ((75, 900), (200, 40), (33, 5000)):
        rows = [(int(rng.integers(0, 4)), int(rng.integers(0, far))) for _ in range(B)]
        rows[B // 2] = (9, far)
        check_attn(ksa, rows, 4, 2, 64, 16, B != 200, B == 75, seed=B)
    rows = [(int(rng.integers(100, 300)), int(rng.integers(1, 3000))) for _ in range(40)]
    check_attn(ksa, rows, 2, 1, 64, 32, True, False, seed=40)


def test_chunk_attn_equal_items_with_a_cut_tail(ksa):
    """Items of one depth that leave a last round half empty: whole ones, then parts."""
    for n, Hkv in ((64 * 37, 5), (64 * 20, 8), (100, 8)):
        check_attn(ksa, [(n, 9000)], Hkv * 4, Hkv, 64, 16, False, False, seed=n)


def test_chunk_attn_repeats_bit_for_bit(ksa):
    """The order in which CTAs finish does not reach the results: split and whole items, 20 runs."""
    for rows, Hq, Hkv in (([(5, 40000)], 8, 2), ([(300, 9000), (64, 20)], 8, 2)):
        cache, q, cu, out, lse = check_attn(ksa, rows, Hq, Hkv, 64, 16, True, True, seed=77)
        ws = torch.zeros(ksa.ksa_chunk_attn_workspace(len(rows), Hq, Hkv, 64,
                                                      cache.table.shape[1] * 16, q.shape[0]),
                         dtype=torch.uint8, device=DEV)
        seq, lse2 = i32([L for _, L in rows]), torch.empty((q.shape[0], Hq), device=DEV)
        for _ in range(20):
            got, _ = cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, workspace=ws, lse=lse2)
            assert torch.equal(got, out[:q.shape[0]]) and torch.equal(lse2, lse)


def test_serving_calls_on_two_streams_at_once(ksa):
    """Calls that overlap, each with its own workspace, give what they give alone."""
    rows = [(3, 30000)]
    cache, q, cu, out, _ = check_attn(ksa, rows, 8, 2, 128, 16, True, True, seed=55)
    seq = i32([30000])
    need = ksa.ksa_chunk_attn_workspace(1, 8, 2, 128, cache.table.shape[1] * 16, 3)
    lanes = [(torch.cuda.Stream(), torch.zeros(need, dtype=torch.uint8, device=DEV),
              torch.empty_like(out)) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, ws, o in lanes:
            cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, out=o, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, o in lanes:
        assert torch.equal(o, out)


def test_serving_calls_allocate_on_the_stream_they_run_on(ksa):
    """A call on a stream that is still busy, with the workspace and outputs left to the binding:
    neither their zeros nor their reuse by the current stream's work may reach it."""
    rows = [(3, 30000), (2, 10)]
    cache, q, cu, out, _ = check_attn(ksa, rows, 8, 2, 128, 16, True, True, seed=56)
    seq = i32([30000, 10])
    T = cache.table.shape[1] * 16
    need = ksa.ksa_chunk_attn_workspace(2, 8, 2, 128, T, 5)
    rng = np.random.default_rng(3)
    table, free, F, pool = page_state(rng, [5, 0, 70], 8, 16, 9)
    want = ref_assign([5, 0, 70], [20, 3, 1], table, free, F, 16, 30, 128, pool)
    tables = [torch.from_numpy(table).to(DEV) for _ in range(2)]
    args = (i32([5, 0, 70]), i32([20, 3, 1]))
    stack, num = torch.from_numpy(free).to(DEV), i32([F])
    side = torch.cuda.Stream()
    long = torch.empty(1 << 29, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for which, t in zip((side, side.cuda_stream), tables):
        with torch.cuda.stream(side):
            for _ in range(40):
                long.fill_(1)
        got, _ = cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, stream=which)
        left = torch.full((1,), -7, dtype=torch.int32, device=DEV)
        torch.cuda.current_stream().synchronize()
        seq2, cu2, slots, pos = ksa.ksa_assign_pages(*args, t, stack, num, 16, 30,
                                                     num_free_out=left, stream=which)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                for n in (need, need, 256, 256, out.numel() * 2)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert all(int(j.min()) == 255 for j in junk)
        assert torch.equal(got, out)
        same_assign((t, left, seq2, cu2, slots, pos, want[6]), want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv,bs,paged", [
    (128, 32, 8, 16, True), (128, 40, 8, 64, False), (64, 32, 8, 32, True), (64, 40, 8, 16, False)])
def test_chunk_attn_ragged_in_pairs(ksa, causal, D, Hq, Hkv, bs, paged):
    """As test_chunk_attn_ragged with so many kv-heads that query tiles go in pairs."""
    check_attn(ksa, EDGES, Hq, Hkv, D, bs, paged, causal, seed=2 * D + Hq + bs, tail=3)


@pytest.mark.parametrize("rows,Hq,Hkv,causal", [
    ([(64 * 40, 9000)], 32, 8, False),                       # two rounds, then a cut tail
    ([(300, 12000), (8, 100), (8, 90)], 64, 8, True),        # deep items cut, short ones not
    ([(0, 50), (700, 6000), (1, 1), (90, 3000)], 32, 8, True)])
def test_chunk_attn_pairs_cut_and_joined(ksa, rows, Hq, Hkv, causal):
    check_attn(ksa, rows, Hq, Hkv, 128, 16, True, causal, seed=91 + len(rows))


def test_chunk_attn_workspace_of_more_tokens_serves_fewer(ksa):
    """One workspace, asked for once with the most tokens, for every smaller call of the batch,
    whatever form it takes."""
    B, Hq, Hkv, T = 3, 32, 8, 4096
    for D in (64, 128):
        sizes = [ksa.ksa_chunk_attn_workspace(B, Hq, Hkv, D, T, n) for n in range(0, 3000, 7)]
        assert sizes == sorted(sizes)


def test_serving_calls_by_both_ways(ksa, monkeypatch):
    """The compiled argument checks and the Python ones make the same calls, and refuse the same
    arguments with the same errors."""
    assert ksa._marshal is not None and ksa._ENTRIES
    N, Hq, Hkv, D, bs = 5, 8, 2, 128, 16
    qkv = randn((N, (Hq + 2 * Hkv) * D), 1)
    q, k, v = (x.view(N, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    pos3 = torch.arange(3 * N, dtype=torch.int32, device=DEV).view(3, N)
    rots = [(ksa.Rotary([1.0 / (i + 1) for i in range(64)]), pos3[:1]),
            (ksa.Rotary([1.0 / (i + 1) for i in range(64)]), pos3[0]),
            (ksa.Rotary([0.5] * 32, [0] * 10 + [1] * 11 + [2] * 11, interleaved=True), pos3)]
    both = []
    for short in (True, False):
        with monkeypatch.context() as m:
            calls = []
            if short:
                for name in ("assign_pages", "release_pages", "rotary_append", "chunk_attn"):
                    real = getattr(ksa._marshal, name)

                    def spy(*a, real=real, name=name):
                        st = real(*a)
                        calls.append((name, st))
                        return st
                    m.setattr(ksa._marshal, name, spy)
            else:
                m.setattr(ksa, "_ENTRIES", {})
            got = []
            table, free, F, pool = page_state(np.random.default_rng(1), [3, 0], 4, bs, 5)
            t, stack, num = torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV), i32([F])
            left, seq, cu = i32([0]), i32([0, 0]), i32([0, 0, 0])
            slots = torch.zeros(N, dtype=torch.int64, device=DEV)
            where = torch.zeros(N, dtype=torch.int32, device=DEV)
            ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
            st = status()
            for out in (left, None):
                ksa.ksa_assign_pages(i32([3, 0]), i32([2, 3]), t, stack, num, bs, N,
                                     num_free_out=out, seq_lens=seq, cu_new=cu, slots=slots,
                                     positions=where, workspace=ws, dev_status=st)
                got += [t.clone(), num.clone(), left.clone(), seq.clone(), cu, slots, where]
            for paged in (True, False):
                for rot, pos in rots:
                    K, V = (torch.zeros((pool if paged else 1, Hkv, bs if paged else 64, D),
                                        dtype=torch.bfloat16, device=DEV) for _ in range(2))
                    to = torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=DEV)
                    call = ksa.ksa_rotary_append_kv_paged if paged else ksa.ksa_rotary_append_kv
                    where2 = slots if paged else torch.arange(N, device=DEV) + 7
                    assert call(q, k, v, pos, where2, K, V, rot, q_out=to) is to
                    got += [to, K, V]
                big = torch.zeros(ksa.ksa_chunk_attn_workspace(2, Hq, Hkv, D, 64, N),
                                  dtype=torch.uint8, device=DEV)
                out = torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=DEV)
                lse = torch.zeros((N, Hq), device=DEV)
                if paged:
                    pair = ksa.ksa_chunk_attn_paged(q, K, V, t, cu, seq, out=out, lse=lse,
                                                    workspace=big, dev_status=st)
                else:
                    pair = ksa.ksa_chunk_attn(q, K.expand(2, -1, -1, -1).contiguous(),
                                              V.expand(2, -1, -1, -1).contiguous(), cu, seq,
                                              ksa.MASK_NONE, 0.5, out, lse, big)
                assert pair[0] is out and pair[1] is lse
                got += [out, lse]
            ksa.ksa_release_pages(seq, i32([1, 0]), t, stack, num, bs, workspace=ws, dev_status=st)
            got += [seq, t, stack, num, st]
            if short:  # every one of these calls was made by it
                assert len(calls) == 2 + 6 + 2 + 1 and all(s == 0 for _, s in calls)
            errors = []
            for bad in (lambda: ksa.ksa_assign_pages(i32([3]), i32([2, 3]), t, stack, num, bs, N),
                        lambda: ksa.ksa_assign_pages(i32([3, 0]), i32([2, 3]), t, stack, num, 8, N,
                                                     left, seq, cu, slots, where, ws),
                        lambda: ksa.ksa_assign_pages(i32([3, 0]), i32([2, 3]), t, stack, num, bs,
                                                     N, left, seq, cu, slots, where, ws[:100]),
                        lambda: ksa.ksa_chunk_attn(q, K, V, cu, seq[:1], out=out, lse=lse,
                                                   workspace=big),
                        lambda: ksa.ksa_chunk_attn(q, K, V, cu[:2], seq[:1], 7, out=out, lse=lse,
                                                   workspace=big),
                        lambda: ksa.ksa_rotary_append_kv(q, k, v, pos3[:2], slots, K, V,
                                                         rots[2][0], q_out=q.contiguous()),
                        lambda: ksa.ksa_release_pages(seq, seq.cpu(), t, stack, num, bs, ws)):
                with pytest.raises(Exception) as e:
                    bad()
                errors.append((type(e.value), str(e.value)))
            torch.cuda.synchronize()
            both.append(([x.clone() for x in got], errors))
    assert len(both[0][0]) == len(both[1][0])
    for a, b in zip(*(x[0] for x in both)):
        assert torch.equal(a, b)
    assert both[0][1] == both[1][1]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [9, 17, 33, 42, 43, 65, 97])
def test_chunk_attn_tiles_with_idle_warps(ksa, D, n):
    """Query tiles that leave some of a stream's warps without rows, over many key tiles, whole
    and cut: such warps keep step with the others."""
    check_attn(ksa, [(n, 2300), (n, 1290), (n, 129)], 8, 2, D, 16, True, True, seed=n)
    check_attn(ksa, [(n, 20011)], 3, 1, D, 32, False, False, seed=n + 1)
    check_attn(ksa, [(n, 2176)] * 40, 24, 8, D, 64, True, False, seed=n + 2)


LONG = [  # B, n, G, D, P pages of 64, L (P * 64 tokens over and over), causal
    (1, 148 * 256, 1, 128, 64, (1 << 20) + 77, False),   # query tiles in pairs, 16 segments and more
    (1, 148 * 256, 1, 128, 64, 65536, False),            # a whole segment, no second one
    (1, 148 * 256, 1, 128, 64, 65537, True),             # one token more
    (1, 148 * 128, 1, 64, 64, 1 << 22, False),           # one tile by one, 64 segments
    (1, 148 * 20, 5, 64, 3, 200003, True),
    (40, 700, 1, 128, 3, 90000, True),
    (148, 1, 8, 128, 64, (1 << 20) + 5, False),          # few rows, whole items
    (296, 2, 2, 64, 5, 300001, True),
    (10, 1, 1, 128, 64, 1 << 23, False),                 # cut, the parts in segments
    (9, 100, 1, 64, 64, 1 << 23, False),
]


@pytest.mark.parametrize("B,n,G,D,P,L,causal", LONG)
def test_chunk_attn_long_sums(ksa, B, n, G, D, P, L, causal):
    """Values with a mean over long rows: no drift with the length.  The rows read the same P pages
    over and over, so that the sums are those over P * 64 tokens, each as often as it is seen.  The
    bounds are those of short rows.  The mean error: over 512 tiles the tensor cores truncate up to
    2.6e-4 of a sum; roundings have no direction, their mean over a row's dims is below 1e-4 (bf16
    weights of 192 tokens or more, 2^-8 / sqrt(12 * 192)), and twice that is allowed.  lse: 512
    additions of a tile's sum and fewer of segments and parts, 2^-24 each."""
    bs, pool = 64, P * 64
    g = torch.Generator(device=DEV)
    g.manual_seed(L % 1000 + D)
    K, V = ((torch.randn((P, 1, bs, D), generator=g, device=DEV) + mean).to(torch.bfloat16)
            for mean in (0.0, 1.0))
    q = torch.randn((B * n, G, D), generator=g, device=DEV).to(torch.bfloat16)
    blocks = -(-L // bs)
    table = (torch.arange(blocks, device=DEV) % P).int()[None].repeat(B, 1)
    lse, st = torch.empty((B * n, G), device=DEV), status()
    mask = ksa.MASK_CAUSAL if causal else ksa.MASK_NONE
    out, _ = ksa.ksa_chunk_attn_paged(q, K, V, table, i32(range(0, B * n + 1, n)), i32([L] * B),
                                      mask, lse=lse, dev_status=st)
    assert int(st) == 0
    k, v = K[:, 0].reshape(pool, D).double(), V[:, 0].reshape(pool, D).double()
    at = torch.arange(pool, device=DEV)
    for b in {0, B // 2, B - 1}:
        for i in {0, n // 2, max(0, n - 129)}:
            rows = torch.arange(i, min(n, i + 129), device=DEV)
            seen = L - n + rows + 1 if causal else torch.full_like(rows, L)
            times = (seen // pool)[:, None] + (at < (seen % pool)[:, None])
            z = torch.einsum("nhd,td->nht", q[b * n + rows].double(), k) * D ** -0.5
            z = z + times.double().log()[:, None]
            want_lse = torch.logsumexp(z, -1)
            w = torch.exp(z - want_lse[..., None])
            want, mag = w @ v, w @ v.abs()
            off = (out[b * n + rows].double() - want).abs()
            assert bool((off <= (HALF + 4e-4) * mag + HALF * want.abs()).all())
            assert float(((out[b * n + rows].double() - want) / mag).mean().abs()) <= 5e-4
            assert float((lse[b * n + rows].double() - want_lse).abs().max()) <= 1e-4


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,Hkv,paged,causal", [
    ([(1, 300), (2, 7), (3, 200), (0, 9)], 4, 2, True, False),      # few rows, whole
    ([(4, 700), (1, 1), (2, 100), (8, 130)], 4, 2, False, True),
    ([(1, 40000)], 8, 2, True, False),                              # few rows, cut
    ([(2, 66000)] * 75, 2, 2, True, True),                          # few rows, in segments
    ([(100, 300), (60, 140)], 2, 2, True, False),                   # one query tile
    ([(90, 20000)], 2, 2, False, True),
    ([(300, 500)] * 20, 16, 8, True, True),                         # pairs
    ([(300, 9000), (280, 30)], 8, 8, False, False),
])
def test_chunk_attn_non_finite_values(ksa, D, rows, Hq, Hkv, paged, causal):
    """NaN and infinities in V of tokens that every query of the row sees: in every form they add up
    as the definition has it (weights are above 0), and reach no other dim, row or head."""
    B, bs = len(rows), 16
    nq, lens = [r[0] for r in rows], [r[1] for r in rows]
    near = [L for _, L in rows if L < 60000] or [2000]
    cache = Cache(near, Hkv, D, bs, paged, seed=D + B)
    if near != lens:  # long rows read the first pages over and over
        L0 = 2000
        table = cache.table[0, :L0 // bs].repeat(B, -(-max(lens) // L0))
        cache.table = table.contiguous()
        cache.rows = [tuple(torch.cat([x] * (lens[0] // L0 + 1), 1)[:, :lens[0]]
                            for x in cache.rows[0])]
    inf, nan = float("inf"), float("nan")
    poison = [(0, 3, inf), (1, 5, -inf), (2, 7, nan), (33, 9, inf), (70, 9, inf), (34, 11, inf),
              (100, 11, -inf), (5, 13, inf), (40, 13, nan), (129, 15, -inf), (6, 33, inf)]
    for b, (n, L) in enumerate(rows[:len(near)]):
        free = L - n if causal else L  # seen by all queries
        for t, d, x in poison:
            if t < min(free, near[b]):
                if paged:
                    cache.V[cache.table[b, t // bs].long(), Hkv - 1, t % bs, d] = x
                else:
                    cache.V[b, Hkv - 1, t, d] = x
                for L1 in range(t, L, 2000 if near != lens else L):
                    cache.rows[b][1][Hkv - 1, L1, d] = x
    if near != lens:
        cache.rows = [cache.rows[0]] * B
    q = randn((sum(nq), Hq, D), 5)
    lse, st = torch.empty((sum(nq), Hq), device=DEV), status()
    out, _ = cache.call(ksa, q, i32(np.concatenate([[0], np.cumsum(nq)])), i32(lens),
                        ksa.MASK_CAUSAL if causal else ksa.MASK_NONE, lse=lse, dev_status=st)
    assert int(st) == 0
    at = 0
    for b, (n, L) in enumerate(rows):
        if n and b in (0, 1, 2, 3, B - 1):
            k, v = cache.rows[b]
            fine = torch.where(torch.isfinite(v.float()), v.float(), 0.0)
            want, want_lse, mag = ref_attn(q[at:at + n], k, fine, n, L, causal, D ** -0.5)
            for x, y in ((inf, inf), (-inf, -inf), (nan, nan)):
                has = v.isnan().any(1) if x != x else (v == x).any(1)  # [Hkv, D]
                has = has.repeat_interleave(Hq // Hkv, 0).expand_as(want)
                if x != x:
                    want = torch.where(has, nan, want)
                else:
                    want = torch.where(has, want + x, want)
            got = out[at:at + n].double()
            assert torch.equal(got.isnan(), want.isnan()), b
            assert torch.equal(got.isinf(), want.isinf())
            assert torch.equal(got[want.isinf()], want[want.isinf()])
            ok = torch.isfinite(want)
            off = (got - want).abs() - (HALF + 4e-4) * mag - HALF * want.abs()
            assert bool((off[ok] <= 1e-30).all())
            assert float((lse[at:at + n].double() - want_lse).abs().max()) <= 1e-4
        at += n


@pytest.mark.parametrize("rows,Hq,Hkv", [([(8, 3)], 2, 1), ([(90, 20)], 1, 1),
                                         ([(300, 200), (300, 40)], 16, 8),
                                         ([(33, 9)] * 3, 1, 1)])
def test_chunk_attn_rows_that_see_nothing_beside_infinities(ksa, rows, Hq, Hkv):
    """More new tokens than cached ones: the first queries see nothing and give 0 and -inf, whatever
    V holds; queries that see an infinity give it."""
    D = 64
    nq, lens = [r[0] for r in rows], [r[1] for r in rows]
    cache = Cache(lens, Hkv, D, 16, False, 5)
    cache.V[:, :, 0, 2] = float("inf")
    cache.V[:, :, 0, 3] = float("nan")
    q = randn((sum(nq), Hq, D), 6)
    out, lse = torch.empty_like(q), torch.empty((sum(nq), Hq), device=DEV)
    cache.call(ksa, q, i32(np.concatenate([[0], np.cumsum(nq)])), i32(lens), ksa.MASK_CAUSAL,
               out=out, lse=lse)
    at = 0
    for n, L in rows:
        none = n - L
        assert bool((out[at:at + none] == 0).all())
        assert bool((lse[at:at + none] == -torch.inf).all())
        assert bool((out[at + none:at + n, :, 2] == torch.inf).all())
        assert bool(out[at + none:at + n, :, 3].isnan().all())
        assert bool(torch.isfinite(out[at + none:at + n, :, 4:].float()).all())
        at += n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,Hkv", [
    ([(2, 200), (1, 50), (3, 129)], 2, 1), ([(1, 30000)], 4, 1), ([(100, 300)], 1, 1),
    ([(90, 20000)], 1, 1), ([(300, 500)] * 20, 8, 8), ([(300, 9000), (260, 129)], 8, 8)])
def test_chunk_attn_scores_of_minus_infinity(ksa, D, rows, Hq, Hkv):
    """A score of -inf weighs nothing; a row of nothing but -inf gives 0 and -inf, also where V holds
    infinities; +inf gives NaN."""
    nq, lens = [r[0] for r in rows], [r[1] for r in rows]
    cache = Cache(lens, Hkv, D, 16, False, 3)
    q = randn((sum(nq), Hq, D), 7).abs() + 0.5
    cu, seq = i32(np.concatenate([[0], np.cumsum(nq)])), i32(lens)
    lse = torch.empty((sum(nq), Hq), device=DEV)
    for b, L in enumerate(lens):  # every third token only
        cache.rows[b][0][:] = torch.where(torch.arange(L, device=DEV)[:, None] % 3 == 0,
                                          cache.rows[b][0].float(), -torch.inf).bfloat16()
        cache.K[b, :, :L] = cache.rows[b][0]
    out, _ = cache.call(ksa, q, cu, seq, ksa.MASK_NONE, lse=lse)
    at = 0
    for b, (n, L) in enumerate(rows):
        k, v = (x[:, ::3] for x in cache.rows[b])
        want, want_lse, mag = ref_attn(q[at:at + n], k, v, n, k.shape[1], False, D ** -0.5)
        off = (out[at:at + n].double() - want).abs() - (HALF + 4e-4) * mag - HALF * want.abs()
        assert bool((off <= 1e-30).all())
        assert float((lse[at:at + n].double() - want_lse).abs().max()) <= 1e-4
        at += n
    for x in (-torch.inf, torch.inf):
        for b, L in enumerate(lens):
            cache.K[b, :, :L] = -torch.inf
            cache.K[b, :, L // 2] = x
            cache.V[b, :, L // 3] = torch.inf
        out, _ = cache.call(ksa, q, cu, seq, ksa.MASK_NONE, lse=lse)
        if x < 0:
            assert bool((out == 0).all()) and bool((lse == -torch.inf).all())
        else:
            assert bool(out.isnan().all()) and bool(lse.isnan().all())


def test_chunk_attn_forms_take_turns_on_one_workspace(ksa):
    """One workspace, as large as the largest call asks for, for whole, cut and segmented calls of
    every form at both head sizes: each gives what it gives on a workspace of its own, and leaves
    the counters and semaphores at zero."""
    calls = []
    for D in (128, 64):
        for rows, Hq, Hkv, T in (([(2, 300), (1, 40)], 8, 2, 0), ([(3, 30000)], 8, 2, 0),
                                 ([(100, 700), (80, 129)], 2, 2, 0), ([(90, 20000)], 2, 2, 0),
                                 ([(300, 500)] * 20, 16, 8, 0), ([(300, 9000), (260, 30)], 8, 8, 0),
                                 ([(2, 66000)] * 75, 2, 2, 2000)):
            nq, lens = [r[0] for r in rows], [r[1] for r in rows]
            cache = Cache([T] if T else lens, Hkv, D, 16, True, D)
            if T:  # the first pages over and over
                cache.table = cache.table[0, :T // 16].repeat(len(rows), lens[0] // T).contiguous()
            q = randn((sum(nq), Hq, D), 9)
            cu, seq = i32(np.concatenate([[0], np.cumsum(nq)])), i32(lens)
            need = ksa.ksa_chunk_attn_workspace(len(rows), Hq, Hkv, D, cache.table.shape[1] * 16,
                                                q.shape[0])
            lse = torch.empty((q.shape[0], Hq), device=DEV)
            own = torch.zeros(need, dtype=torch.uint8, device=DEV)
            out, _ = cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, lse=lse, workspace=own)
            calls.append((cache, q, cu, seq, out, lse, need))
    ws = torch.zeros(max(c[-1] for c in calls), dtype=torch.uint8, device=DEV)
    marks = 256 + 4 * 3 * torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(4)
    for _ in range(3):
        for i in rng.permutation(len(calls)):
            cache, q, cu, seq, out, lse, _ = calls[i]
            lse2, st = torch.empty_like(lse), status()
            got, _ = cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, lse=lse2, workspace=ws,
                                dev_status=st)
            assert torch.equal(got, out) and torch.equal(lse2, lse) and int(st) == 0
            assert not bool(ws[:marks].any())


@pytest.mark.parametrize("rows,tail,Hq,Hkv", [
    ([(1, 1000 + 37 * b) for b in range(31)] + [(300, 2100)], 0, 8, 2),  # decode rows and a chunk
    ([(1, 129 * (b + 1)) for b in range(20)] + [(512, 512), (1, 3)], 0, 32, 8),
    ([(1, 700 + b) for b in range(16)], 500, 8, 2),                      # a padded token axis
    ([(1, 700 + b) for b in range(16)], 8000, 32, 8),
    ([(0, 0), (5, 5), (0, 900), (2, 1500)], 100, 16, 2)])
def test_chunk_attn_mixed_batches_and_padded_axes(ksa, rows, tail, Hq, Hkv):
    check_attn(ksa, rows, Hq, Hkv, 128, 16, True, True, seed=len(rows) + tail, tail=tail)


@pytest.mark.parametrize("N", [8, 90, 2000])
def test_captured_chunk_attn_follows_the_lengths(ksa, N):
    """A captured call whose rows change from replay to replay, from all tokens in one row to one
    token in each, and to none: what an eager call gives."""
    B, Hq, Hkv, D, bs = 4, 8, 4, 64, 16
    cache = Cache([3000] * B, Hkv, D, bs, True, 11)
    q = randn((N, Hq, D), 12)
    cu, seq, st = i32([0] * (B + 1)), i32([0] * B), status()
    out, lse = torch.empty_like(q), torch.empty((N, Hq), device=DEV)
    ws = torch.zeros(ksa.ksa_chunk_attn_workspace(B, Hq, Hkv, D, cache.table.shape[1] * bs, N),
                     dtype=torch.uint8, device=DEV)
    call = lambda: cache.call(ksa, q, cu, seq, ksa.MASK_CAUSAL, out=out, lse=lse, workspace=ws,
                              dev_status=st)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    n = N // 4
    for nq, lens in (([N, 0, 0, 0], [3000, 5, 0, 7]), ([1, 1, 1, 1], [1, 3000, 128, 129]),
                     ([0, 0, 0, 0], [9, 9, 9, 9]), ([n, 0, n, 1], [n, 40, 2999, 2]),
                     ([0, 0, 1, N - 1], [0, 0, 777, 3000])):
        cu.copy_(i32(np.concatenate([[0], np.cumsum(nq)])))
        seq.copy_(i32(lens))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for b, (m, L) in enumerate(zip(nq, lens)):
            k, v = (x[:, :L] for x in cache.rows[b])
            want, _, mag = ref_attn(q[at:at + m], k, v, m, L, True, D ** -0.5)
            off = (out[at:at + m].double() - want).abs() - (HALF + 4e-4) * mag - HALF * want.abs()
            assert bool((off <= 1e-30).all()), (nq, b)
            at += m
        assert bool((out[at:] == 5.0).all()) and int(st) == 0
    del graph


def test_serving_calls_refuse_numbers_past_32_bits(ksa):
    """Numbers that the library takes as 32 bits are not cut off: 2^32 + 16 is no block size."""
    far = 1 << 32
    table, free, one = i32([[0, 1]]), i32([0, 1, 2]), i32([1])
    assign = lambda **kw: ksa.ksa_assign_pages(**{**dict(
        ctx_lens=one, new_lens=one, block_table=table, free_pages=free, num_free=one,
        block_size=16, num_tokens=2), **kw})
    q, K = torch.zeros((1, 1, 64), device=DEV).bfloat16(), torch.zeros((1, 1, 4, 64),
                                                                       device=DEV).bfloat16()
    for call in (lambda: assign(block_size=far + 16), lambda: assign(num_tokens=far + 2),
                 lambda: assign(num_tokens=-far - 2),
                 lambda: ksa.ksa_release_pages(one, one, table, free, one, far + 16),
                 lambda: ksa.ksa_chunk_attn(q, K, K, i32([0, 1]), one, mask=far + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert table.tolist() == [[0, 1]] and free.tolist() == [0, 1, 2] and int(one) == 1
