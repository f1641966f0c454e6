"""Token-by-token generation on the GPU, the edges: weights that cancel, columns and rows that no sequence owns,
malformed row tables, captured calls whose contexts are cut into pieces, empty batches, values that are not
finite behind a row's last token, pages outside the cache.  Bounds as in test_decode_gpu: u = 2^-24 (fp32),
2^-8 (bf16)."""
import numpy as np
import pytest

from oracle import decode as od
from test_decode_gpu import SCALE, U32, UBF, batch, dev, host, rounded, starts, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import tree_packed_chunkwise_b200 as t
    t.lib()
    return t


def i32(a):
    return dev(np.asarray(a, np.int32))


def new_status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------ weights of the softmax
@pytest.mark.parametrize("H,m", [(5, 1), (16, 1), (16, 2), (16, 4), (40, 1)])
@pytest.mark.parametrize("L", [2, 7, 40, 129, 300])
def test_attention_of_cancelling_tokens(tpc, H, m, L):
    """Neighbouring tokens have opposite latents, so that the outputs are differences of weights.
    A query has one value that is not zero: scores are single products of bf16 values, exact in fp32.  A weight is
    then off by less than 2^-14 (scaling, exponential, sums, as in test_decode_gpu) and by the rounding of the two
    bf16 values that stand for it in the product, u^2 = 2^-16; the output rounds once more to bf16."""
    import torch
    rng = np.random.default_rng(100 * H + L + m)
    page, kv = 16, L + m - 1
    table = rng.permutation(-(-kv // page)).astype(np.int32)[None]
    x = rng.normal(size=(table.shape[1] * page, 576))
    x[1::2, 1:512] = -x[::2, 1:512]
    x[:, 0] = rng.uniform(-1, 1, len(x))
    cache = torch.empty(table.shape[1], page, 576, dtype=torch.bfloat16, device="cuda")
    cache[i32(table[0]).long()] = dev(x.reshape(cache.shape), torch.bfloat16)
    q = np.zeros((m, H, 576))
    q[:, :, 0] = rng.uniform(0.5, 1.5, (m, H))
    qa = dev(q, torch.bfloat16)
    status = new_status()
    o, lse = tpc.tpc_latent_attn(qa, cache, i32(table), i32([kv]), 1.0, row_start=i32([0, m]), status=status)
    assert status.item() == 0
    ref, lref, oa, _ = od.attention(host(qa), host(cache), table, [kv], 1.0, [0, m])
    within(host(o), ref, UBF * np.abs(ref) + (2.0 ** -14 + 2.0 ** -16 + kv * U32) * oa, "o")
    within(host(lse), lref, 2.0 ** -18 + kv * U32 + 4 * U32 * np.abs(lref), "lse")


# ------------------------------------------------------------------------------------ rows of other sequences and of none
@pytest.mark.parametrize("H,m", [(5, 1), (5, 3), (16, 1), (24, 1), (24, 2), (40, 1), (5, 13)])
def test_attention_rows_that_a_unit_does_not_own(tpc, H, m):
    """The bits of a sequence's outputs depend on its own rows alone, whatever the rows behind the last sequence
    hold and whatever the next sequence asks.  Scores rise along the context, slowly for every second sequence and
    by more than the running maximum's slack in every tile for the others; the shares are several tiles long."""
    import torch
    rng = np.random.default_rng(H + m)
    page, kv, extra, B = 64, 700, 16, 120
    cache, _ = rounded(rng, 11, page, 576, dtype=torch.bfloat16)
    cache[:, :, 0] = torch.arange(11 * page, device="cuda").view(11, page).bfloat16() / 4
    table = i32(np.broadcast_to(np.arange(11), (B, 11)))
    mine = (torch.arange(B, device="cuda") % 2 == 0).repeat_interleave(m)
    qa, _ = rounded(rng, B * m + extra, H, 576, dtype=torch.bfloat16, s=0.05)
    qa[:, :, 0] = 8.0
    qa[:B * m][mine, :, 0] = 0.02
    status = new_status()
    got = []
    for fill in (None, 0.0, 300.0, float("inf"), float("-inf"), float("nan")):
        q = qa.clone()
        if fill is not None:
            q[B * m:] = fill
            q[:B * m][~mine] *= -1.0
        o = torch.full((len(q), H, 512), -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((len(q), H), -7.0, device="cuda")
        tpc.tpc_latent_attn(q, cache, table, i32([kv] * B), 1.0, row_start=i32(np.arange(B + 1) * m), o=o, lse=lse, status=status)
        assert bool((o[B * m:] == -7).all()) and bool((lse[B * m:] == -7).all())
        got.append((o[:B * m][mine], lse[:B * m][mine]))
    assert status.item() == 0 and bool(torch.isfinite(got[0][0].float()).all())
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


# ------------------------------------------------------------------------------------ malformed row tables
@pytest.mark.parametrize("start", [[0, 1, 2, 9], [-4, 1, 2, 3], [3, 2, 1, 0], [0, 2, 1, 3], [2 ** 31 - 1, 0, 1, 3], [0, -2 ** 31 + 1, 2 ** 31 - 1, 3],
                                   [0, 1, 3, 4], [0, 0, 7, 3]])
def test_bad_row_starts_are_skipped_and_reported_by_every_call(tpc, start):
    """A sequence whose rows are not within 0 .. n_rows, or decrease, has no rows: append leaves its cached tokens
    and absorb its outputs as they were, the others are right (unless two sequences claim a row), and each call by
    itself sets the status."""
    import torch
    rng = np.random.default_rng(abs(start[0]) % 97 + start[-1])
    H, n, page, kv = 3, 3, 16, [20, 9, 31]
    table = rng.permutation(6).reshape(3, 2).astype(np.int32)
    good = [b for b in range(3) if 0 <= start[b] <= start[b + 1] <= n]
    claims = [[b for b in good if start[b] <= t < start[b + 1]] for t in range(n)]
    c, c64 = rounded(rng, n, 512, dtype=torch.bfloat16)
    kr, k64 = rounded(rng, n, 64, dtype=torch.bfloat16)
    cache, before = rounded(rng, 6, page, 576, dtype=torch.bfloat16)
    status = new_status()
    tpc.tpc_latent_append(cache, i32(table), i32(kv), c, kr, row_start=i32(start), status=status)
    assert status.item() == 7
    want, free = before.copy(), np.zeros((6, page), bool)
    for b in good:
        for i in range(start[b + 1] - start[b]):
            p, t = kv[b] - (start[b + 1] - start[b]) + i, start[b] + i
            at = table[b, p // page], p % page
            if claims[t] == [b]:
                want[at] = np.concatenate([c64[t], od.rotate(k64[t], p)])
            else:
                free[at] = True
    x = host(cache)
    assert np.array_equal(x[..., :512][~free], want[..., :512][~free])
    tol = UBF * np.abs(want[..., 512:]) + 2.0 ** -19 * np.abs(k64).max()
    within(x[..., 512:][~free], want[..., 512:][~free], tol[~free], "rotary key")

    q, q64 = rounded(rng, n, H, 192, dtype=torch.bfloat16)
    w_b, w64 = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
    qa = torch.full((n, H, 576), -7.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    tpc.tpc_latent_absorb(q, w_b, i32(kv), row_start=i32(start), qa=qa, status=status)
    assert status.item() == 7
    x = host(qa)
    for t in range(n):
        if not claims[t]:
            assert (x[t] == -7).all(), t
        elif len(claims[t]) == 1:
            b = claims[t][0]
            ref, mag = od.absorb(q64[t:t + 1], w64, [kv[b] - (start[b + 1] - start[b]) + t - start[b] + 1])
            tol = UBF * np.abs(ref) + np.where(np.arange(576) < 512, 140 * U32, 2.0 ** -19) * mag
            within(x[t:t + 1], ref, tol, t)


def test_absorb_of_bad_row_starts_in_large_batches(tpc):
    """One decreasing pair among 300 sequences of several tiles: every other row is as in the sound batch."""
    import torch
    rng = np.random.default_rng(3)
    H, m = 5, rng.integers(0, 4, 300)
    m[[40, 41, 200]] = [2, 1, 3]
    start = starts(m)
    n = int(start[-1]) + 5
    kv = i32(rng.integers(5, 9000, 300))
    q, _ = rounded(rng, n, H, 192, dtype=torch.bfloat16)
    w_b, _ = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
    status, res = new_status(), []
    bad = start.copy()
    bad[41] += 10 ** 6  # sequence 40 leaves the rows, sequence 41 decreases
    for s in (start, bad):
        qa = torch.full((n, H, 576), -7.0, dtype=torch.bfloat16, device="cuda")
        status.zero_()
        tpc.tpc_latent_absorb(q, w_b, kv, row_start=i32(s), qa=qa, status=status)
        res.append(qa)
        assert status.item() == (0 if s is start else 7)
    lost = np.zeros(n, bool)
    lost[start[40]:start[42]] = True
    assert torch.equal(res[0][dev(~lost)], res[1][dev(~lost)])
    assert bool((res[1][dev(lost)] == -7).all()) and bool((res[1][n - 5:] == -7).all())


# ------------------------------------------------------------------------------------ contexts cut into pieces
def test_capture_and_replay_with_cut_contexts(tpc):
    """A captured append and attention (and its joining launch), replayed with lengths that move between one
    tile, few pieces and more than 32 pieces, against the same calls outside a graph and the definition."""
    import torch
    rng = np.random.default_rng(51)
    page, most = 64, 6100
    per = -(-most // page)
    lengths = [[1, 50, 128, 0, 7], [6000, 0, 0, 0, 0], [3000, 130, 0, 6100, 64], [129, 257, 600, 40, 5000], [0, 0, 0, 0, 0], [0, 0, 6100, 1, 0]]
    for H in (16, 24, 40):  # 16, 32 and 64 columns a tile
        table = rng.permutation(5 * per).reshape(5, per).astype(np.int32)
        cache, _ = rounded(rng, 5 * per, page, 576, dtype=torch.bfloat16)
        tab, scratch, status = i32(table), tpc.latent_attn_scratch(H), new_status()
        buf = dict(kv=i32(lengths[0]), qa=rounded(rng, 5, H, 576, dtype=torch.bfloat16)[0], x=rounded(rng, 5, 576, dtype=torch.bfloat16)[0])

        def call(b, ch, sc):
            tpc.tpc_latent_append(ch, tab, b["kv"], b["x"][:, :512], b["x"][:, 512:], status=status)
            return tpc.tpc_latent_attn(b["qa"], ch, tab, b["kv"], SCALE, scratch=sc, status=status)

        twin = cache.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(buf, twin, scratch)
        torch.cuda.current_stream().wait_stream(side)
        twin.copy_(cache)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call(buf, cache, scratch)
        for kv in lengths + lengths[::-1]:
            new = dict(kv=i32(kv), qa=rounded(rng, 5, H, 576, dtype=torch.bfloat16)[0], x=rounded(rng, 5, 576, dtype=torch.bfloat16)[0])
            for k in buf:
                buf[k].copy_(new[k])
            graph.replay()
            want = call(new, twin, tpc.latent_attn_scratch(H))
            assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(cache, twin), kv
        del graph
        q64 = host(buf["qa"])
        ref, lref, oa, sa = od.attention(q64, host(cache), table, lengths[0], SCALE)
        tol = UBF * np.abs(ref) + (2 * 640 * U32 * sa[..., None] + 2.0 ** -14 + 2.0 ** -16 + most * U32) * oa
        within(host(outs[0]), ref, tol, "o")
        assert status.item() == 0


def test_attention_bad_tables_of_cut_contexts(tpc):
    """Bad entries anywhere in a long context, and lengths beyond its table, among contexts that shares cut: the
    status is set and the other sequences are right."""
    import torch
    rng = np.random.default_rng(52)
    page, per, H, kv = 64, 40, 16, [2500, 2560, 700]
    cache, c64 = rounded(rng, 3 * per, page, 576, dtype=torch.bfloat16)
    qa, q64 = rounded(rng, 3, H, 576, dtype=torch.bfloat16)
    table = rng.permutation(3 * per).reshape(3, per).astype(np.int32)
    ref, lref, oa, sa = od.attention(q64, c64, table, kv, SCALE)
    tol = UBF * np.abs(ref) + (2 * 640 * U32 * sa[..., None] + 2.0 ** -14 + 2.0 ** -16 + 2560 * U32) * oa
    for at, entry, length in ((0, 3 * per, 2560), (17, -1, 2560), (39, 2 ** 31 - 1, 2560), (20, -2 ** 31, 2560), (0, table[1, 0], 2561),
                              (0, table[1, 0], 2 ** 31 - 1)):
        bad = table.copy()
        bad[1, at] = entry
        status = new_status()
        o, lse = tpc.tpc_latent_attn(qa, cache, i32(bad), i32([kv[0], length, kv[2]]), SCALE, status=status)
        assert status.item() == 7, (at, entry, length)
        for b in (0, 2):
            within(host(o)[b], ref[b], tol[b], "o")
            within(host(lse)[b], lref[b], 640 * U32 * sa[b] + 2.0 ** -18 + 2560 * U32 + 4 * U32 * np.abs(lref[b]), "lse")


@pytest.mark.parametrize("start", [[0, 2, 1, 3], [-4, 1, 2, 3], [0, 1, 2, 9], [2 ** 31 - 1, 0, 1, 3], [0, -2 ** 31 + 1, 2 ** 31 - 1, 3], [3, 2, 1, 0]])
def test_attention_bad_row_starts_of_cut_contexts(tpc, start):
    """Malformed row tables over long contexts: reported, rows of no sequence and the memory around the outputs
    stay as they were, rows of one sound sequence are right."""
    import torch
    rng = np.random.default_rng(53)
    page, per, H, n, kv = 64, 50, 40, 3, [3000, 2 ** 31 - 1, 129]
    cache, c64 = rounded(rng, 3 * per, page, 576, dtype=torch.bfloat16)
    qa, q64 = rounded(rng, n, H, 576, dtype=torch.bfloat16)
    table = rng.permutation(3 * per).reshape(3, per).astype(np.int32)
    o = torch.full((9, H, 512), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, H), -7.0, device="cuda")
    status = new_status()
    tpc.tpc_latent_attn(qa, cache, i32(table), i32(kv), SCALE, row_start=i32(start), o=o[3:6], lse=lse[3:6], status=status)
    assert status.item() == 7
    for t in (o, lse):
        assert bool((t[:3] == -7).all()) and bool((t[6:] == -7).all())
    good = [b for b in range(3) if 0 <= start[b] <= start[b + 1] <= n]
    for t in range(n):
        owner = [b for b in good if start[b] <= t < start[b + 1]]
        if not owner:
            assert bool((o[3 + t] == -7).all())
        elif len(owner) == 1 and kv[owner[0]] <= per * page:
            b = owner[0]
            seen = kv[b] - (start[b + 1] - start[b]) + 1 + t - start[b]
            ref, lref, oa, sa = od.attention(q64[t:t + 1], c64, table[b:b + 1], [seen], SCALE)
            tol = UBF * np.abs(ref) + (2 * 640 * U32 * sa[..., None] + 2.0 ** -14 + 2.0 ** -16 + 3000 * U32) * oa
            within(host(o)[3 + t:4 + t], ref, tol, "o")


# ------------------------------------------------------------------------------------ nothing to do
@pytest.mark.parametrize("seqs", [0, 3])
def test_empty_batches(tpc, seqs):
    """No live sequence, and sequences without a new row: every call returns its empty result and touches nothing."""
    import torch
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    H, status = 2, new_status()
    for start in ([None] if seqs == 0 else []) + [i(seqs + 1)]:
        cache = z(4, 16, 576) + 3
        kw = dict(row_start=start, status=status)
        tpc.tpc_latent_append(cache, i(seqs, 2), i(seqs), z(0, 512), z(0, 64), **kw)
        assert bool((cache == 3).all())
        assert tpc.tpc_latent_absorb(z(0, H, 192), z(512, 512), i(seqs), **kw).shape == (0, H, 576)
        o, lse = tpc.tpc_latent_attn(z(0, H, 576), cache, i(seqs, 2), i(seqs), SCALE, **kw)
        assert o.shape == (0, H, 512) and lse.shape == (0, H)
        assert tpc.tpc_latent_expand(z(0, H, 512), z(512, 512), status=status).shape == (0, H, 128)
        x, state = z(0, H, 64), z(4, H, 64, 64, t=torch.float32) + 3
        src = torch.arange(seqs, dtype=torch.int32, device="cuda")
        assert tpc.tpc_kda_step(state, src, x, x, x, x, z(0, H), **kw).shape == (0, H, 64)
        assert bool((state == 3).all())
    # rows that belong to no sequence
    n = 2
    cache, start = z(4, 16, 576) + 3, i(1)
    qa, o = z(n, H, 576) + 3, z(n, H, 512) + 3
    lse = z(n, H, t=torch.float32) + 3
    tpc.tpc_latent_append(cache, i(0, 2), i(0), z(n, 512), z(n, 64), row_start=start, status=status)
    tpc.tpc_latent_absorb(z(n, H, 192), z(512, 512), i(0), row_start=start, qa=qa, status=status)
    tpc.tpc_latent_attn(z(n, H, 576), cache, i(0, 2), i(0), SCALE, row_start=start, o=o, lse=lse, status=status)
    for t in (cache, qa, o, lse):
        assert bool((t == 3).all())
    assert status.item() == 0


# ------------------------------------------------------------------------------------ waits that run out
def test_waits_that_run_out_leave_the_device_usable(tpc):
    """With a limit of zero every tensor-core kernel gives up at its first wait, with copies and perhaps products in
    flight: it records the timeout, writes nothing outside its outputs, and the next calls are right."""
    import torch
    rng = np.random.default_rng(61)
    guard = 4096

    def framed(*s, t=torch.bfloat16):
        """A tensor inside a larger one, and the larger one."""
        n = int(np.prod(s))
        whole = torch.full((n + 2 * guard,), -7.0, dtype=t, device="cuda")
        return whole[guard:guard + n].view(*s), whole

    def untouched(whole):
        return bool((whole[:guard] == -7).all()) and bool((whole[-guard:] == -7).all())

    calls = []
    for H, m, kv in ((16, 1, 20000), (16, 2, 5000), (16, 40, 3000), (5, 3, 100), (40, 1, 64)):
        B = 6
        table, n_pages = batch(rng, [kv] * B, 64)
        cache, _ = rounded(rng, n_pages, 64, 576, dtype=torch.bfloat16)
        qa, _ = rounded(rng, B * m, H, 576, dtype=torch.bfloat16)
        args = (qa, cache, i32(table), i32([kv] * B), SCALE)
        start = i32(np.arange(B + 1) * m)
        calls.append(([((B * m, H, 512), torch.bfloat16), ((B * m, H), torch.float32)],
                      lambda out, st, args=args, start=start: tpc.tpc_latent_attn(*args, row_start=start, o=out[0], lse=out[1], status=st)))
    for n, H in ((1, 16), (500, 16), (3000, 16), (130, 3)):
        q, _ = rounded(rng, n, H, 192, dtype=torch.bfloat16)
        o, _ = rounded(rng, n, H, 512, dtype=torch.bfloat16)
        w_b, _ = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
        kv = i32(rng.integers(1, 9000, n))
        calls.append(([((n, H, 576), torch.bfloat16)], lambda out, st, a=(q, w_b, kv): tpc.tpc_latent_absorb(*a, qa=out[0], status=st)))
        calls.append(([((n, H, 128), torch.bfloat16)], lambda out, st, a=(o, w_b): tpc.tpc_latent_expand(*a, out=out[0], status=st)))

    def run(code):
        res = []
        for shapes, call in calls:
            frames, status = [framed(*s, t=t) for s, t in shapes], new_status()
            call([f[0] for f in frames], status)
            torch.cuda.synchronize()
            assert status.item() == code and all(untouched(f[1]) for f in frames)
            res.append([f[0] for f in frames])
        return res

    before = run(0)
    normal = tpc.tpc_debug_wait_limit(0)
    try:
        run(8)
        run(8)
    finally:
        assert tpc.tpc_debug_wait_limit(normal) == 0
    assert normal == 2_000_000_000
    after = run(0)
    for a, b in zip(before, after):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("H,m", [(5, 3), (16, 2), (16, 3), (16, 4), (16, 9), (3, 70), (40, 150)])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_attention_does_not_see_later_tokens(tpc, H, m, value):
    """A later token of the same run that is not finite (in one dimension, in all, in its rotary key) leaves the
    rows before it as they are; a query that is not finite leaves the other rows as they are."""
    import torch
    rng = np.random.default_rng(7 * H + m)
    page, kv = 64, 300
    table = rng.permutation(5).astype(np.int32)[None]
    clean, _ = rounded(rng, 5, page, 576, dtype=torch.bfloat16)
    qa, _ = rounded(rng, m, H, 576, dtype=torch.bfloat16)
    start, bad = i32([0, m]), float(value)

    def call(cache, q):
        status = new_status()
        o, lse = tpc.tpc_latent_attn(q, cache, i32(table), i32([kv]), SCALE, row_start=start, status=status)
        assert status.item() == 0
        return o, lse

    def token(cache, j):
        return cache[int(table[0, j // page]), j % page]

    o0, l0 = call(clean, qa)
    assert bool(torch.isfinite(o0.float()).all())
    for row in {1, m // 2, m - 1}:       # the row at kv - m + row and all behind it see the token
        for dims in (slice(0, 512), slice(37, 38), slice(511, 512), slice(540, 541), slice(0, 576)):
            cache = clean.clone()
            token(cache, kv - m + row)[dims] = bad
            o, lse = call(cache, qa)
            assert torch.equal(o[:row], o0[:row]) and torch.equal(lse[:row], l0[:row]), (row, dims)
            if dims.stop - dims.start > 64 and value == "nan":
                assert bool(torch.isnan(o[row:].float()).all()) and bool(torch.isnan(lse[row:]).all())
    cache = clean.clone()                # several of them
    for j in range(kv - m + 1, kv):
        token(cache, j)[j % 512] = bad
    o, lse = call(cache, qa)
    assert torch.equal(o[0], o0[0]) and torch.equal(lse[0], l0[0])
    for row in {0, m // 2, m - 1}:       # a query: the other rows' tokens stay in their sums
        q = qa.clone()
        q[row, :, 5] = bad
        o, lse = call(clean, q)
        rest = torch.arange(m, device="cuda") != row
        assert torch.equal(o[rest], o0[rest]) and torch.equal(lse[rest], l0[rest]), row


# ------------------------------------------------------------------------------------ races between written pages
def test_append_of_a_long_run_is_checked_in_its_time(tpc):
    """A prompt of 100,000 tokens in 16-token pages, 6,250 written pages that are all compared: with a status word
    the append takes at most three quarters longer than without."""
    import torch
    n, page = 100_000, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(n // page, generator=g, device="cuda").int()[None]
    cache = torch.zeros(n // page, page, 576, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(n, 576, generator=g, device="cuda").bfloat16()
    kv, start, status = i32([n]), i32([0, n]), new_status()

    def us(**kw):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            tpc.tpc_latent_append(cache, table, kv, x[:, :512], x[:, 512:], row_start=start, **kw)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times)[2]

    plain, checked = us(), us(status=status)
    assert status.item() == 0
    assert checked < 1.75 * plain, (plain, checked)
    # the same page at both ends of the run, and next to each other
    for a, b in ((0, n // page - 1), (3, 4), (17, 4000)):
        t = table.clone()
        t[0, a] = t[0, b]
        status.zero_()
        tpc.tpc_latent_append(cache, t, kv, x[:, :512], x[:, 512:], row_start=start, status=status)
        assert status.item() == 7, (a, b)


@pytest.mark.parametrize("m", [[1] * 70, [40] * 70, [1] * 31 + [900] + [1] * 38, [0] * 40 + [300, 0, 300] + [1] * 40, [17, 0, 1, 500]])
def test_append_races_between_any_two_sequences(tpc, m):
    """Sequences of few and of many pages: a page that any two of them write, or one twice, is found wherever it
    stands; pages that are shared but not written are none."""
    import torch
    rng = np.random.default_rng(sum(m))
    page, B, n = 16, len(m), sum(m)
    kv = [x + int(rng.integers(0, 40)) if x else 33 for x in m]
    per = max(-(-L // page) for L in kv)
    x = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(B * per, page, 576, dtype=torch.bfloat16, device="cuda")
    sound = rng.permutation(B * per).reshape(B, per).astype(np.int32)
    written = [(b, p) for b in range(B) if m[b] for p in range((kv[b] - m[b]) // page, -(-kv[b] // page))]
    kept = [(b, p) for b in range(B) for p in range(0, (kv[b] - m[b]) // page)]

    def status_of(t):
        status = new_status()
        tpc.tpc_latent_append(cache, i32(t), i32(kv), x[:, :512], x[:, 512:], row_start=i32(starts(m)), status=status)
        return status.item()

    assert status_of(sound) == 0
    shared = sound.copy()
    for b, p in kept:
        shared[b, p] = sound[kept[0]]
    assert status_of(shared) == 0
    pairs = [rng.choice(len(written), 2, replace=False) for _ in range(12)] + [(0, len(written) - 1), (len(written) - 2, len(written) - 1)]
    for i, j in pairs:
        t = sound.copy()
        t[written[i]] = t[written[j]]
        assert status_of(t) == 7, (written[i], written[j])


# ------------------------------------------------------------------------------------ pages outside the cache
@pytest.mark.parametrize("entry", [-1, 48, 2 ** 31 - 1])
@pytest.mark.parametrize("H", [16, 24, 40])
def test_attention_of_pages_outside_the_cache_reads_no_other_page(tpc, entry, H):
    """An entry outside the cache, with or without a status word: the outputs of its sequence are unspecified, but
    they do not depend on what other sequences' pages hold."""
    import torch
    rng = np.random.default_rng(H)
    cache, _ = rounded(rng, 48, 64, 576, dtype=torch.bfloat16)
    qa, _ = rounded(rng, 1, H, 576, dtype=torch.bfloat16)
    table = np.arange(20, 40, dtype=np.int32)[None]
    table[0, [0, 7, 19]] = entry
    rest = torch.ones(48, dtype=torch.bool, device="cuda")
    rest[20:40] = False
    rest[[20, 27, 39]] = True
    got = []
    for fill in (1.0, -2.0, float("nan")):
        cache[rest] = fill
        got.append(tpc.tpc_latent_attn(qa, cache, i32(table), i32([1250]), SCALE))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
