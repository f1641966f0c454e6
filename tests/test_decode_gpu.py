"""Token-by-token generation on the GPU (recurrent KDA step, latent cache append, absorb, attention,
expand) against the fp64 oracle.  Bounds are sums of half-step roundings (u = 2^-24 fp32, 2^-8 bf16) times
the magnitudes the oracle returns:
* a dot product of d terms in fp32 is off by at most d u times the sum of magnitudes, an update by a few u;
* the softmax: a score is off by ds = 640 u scale sum |q||k|, a weight by exp(ds) - 1 and its bf16 rounding,
  the exponential and the sums by less than 2^-14 in all; outputs round once more to bf16.
"""
import numpy as np
import pytest

from oracle import decode as od

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def tpc():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import tree_packed_chunkwise_b200 as t
    t.lib()
    return t


def dev(a, dtype=None):
    import torch
    t = torch.as_tensor(np.ascontiguousarray(a))
    if dtype is not None:
        t = t.to(dtype)
    elif t.dtype == torch.int64:
        t = t.to(torch.int32)
    return t.cuda()


def host(t):
    return t.double().cpu().numpy()


def rounded(rng, *shape, dtype, s=1.0):
    """A device tensor of dtype and its values in fp64."""
    t = dev(s * rng.normal(size=shape), dtype)
    return t, host(t)


def within(x, ref, tol, what):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(x - ref) <= tol) & ~(x == ref)  # a NaN is bad, equal infinities are not
    i = np.argmax(bad) if bad.size else 0
    assert not bad.any(), (what, int(bad.sum()), np.unravel_index(i, x.shape), x.flat[i], ref.flat[i],
                           np.broadcast_to(tol, x.shape).flat[i])


def starts(m):
    return np.concatenate([[0], np.cumsum(m)]).astype(np.int32)


# ------------------------------------------------------------------------------------ KDA step
def step_case(rng, seqs, H, d, dtype, m=None, extra_rows=0, slots=None, fork=False):
    import torch
    m = np.ones(seqs, int) if m is None else np.asarray(m)
    n = int(m.sum()) + extra_rows
    c = dict(m=m, n=n, start=None if (m == 1).all() and not extra_rows else starts(m))
    c["q"], c["q64"] = rounded(rng, n, H, d, dtype=dtype)
    k = rng.normal(size=(n, H, d))
    c["k"] = dev(k / np.linalg.norm(k, axis=-1, keepdims=True), dtype)
    c["v"], c["v64"] = rounded(rng, n, H, d, dtype=dtype)
    c["g"] = dev(-0.1 * np.log1p(np.exp(rng.normal(size=(n, H, d)))), dtype)
    c["beta"] = dev(1 / (1 + np.exp(-rng.normal(size=(n, H)))), dtype)
    for x in ("k", "g", "beta"):
        c[x + "64"] = host(c[x])
    slots = slots or (2 * seqs + 3 if fork else seqs + 2)
    c["state"], c["state64"] = rounded(rng, slots, H, d, d, dtype=torch.float32)
    perm = rng.permutation(slots)
    if fork:
        c["src"] = perm[rng.integers(0, max(1, seqs // 2), seqs)].astype(np.int32)
        c["dst"] = perm[slots - seqs:].astype(np.int32)
    else:
        c["src"], c["dst"] = perm[:seqs].astype(np.int32), None
    return c


def check_step(tpc, c, out_dtype=None, d=None, **kw):
    import torch
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = c["q"].shape[2]
    out_dtype = out_dtype or c["q"].dtype
    o = torch.full(c["q"].shape, -7.0, dtype=out_dtype, device="cuda")
    got = tpc.tpc_kda_step(c["state"], dev(c["src"]), c["q"], c["k"], c["v"], c["g"], c["beta"],
                           dst=None if c["dst"] is None else dev(c["dst"]),
                           row_start=None if c["start"] is None else dev(c["start"]), o=o, status=status, **kw)
    torch.cuda.synchronize()
    assert got is o and status.item() == 0
    ref, new, oa, na = od.kda_step(c["state64"], c["src"], c["src"] if c["dst"] is None else c["dst"], c["q64"],
                                   c["k64"], c["v64"], c["g64"], c["beta64"], c["start"])
    T = max(1, int(c["m"].max()) if len(c["m"]) else 1)
    gam = (T * (d + 12) + d) * U32
    own = ~np.isnan(ref)
    tol = gam * np.where(own, oa, 0) + (UBF * np.abs(ref) if out_dtype == torch.bfloat16 else 0)
    x = host(o)
    within(x[own], ref[own], tol[own], "o")
    assert (x[~own] == -7.0).all()  # rows of no sequence and of padding entries
    within(host(c["state"]), new, gam * na, "state")
    touched = np.zeros(len(new), bool)
    for b, s in enumerate(c["src"]):
        if s >= 0:
            touched[s if c["dst"] is None else c["dst"][b]] = True
    assert np.array_equal(host(c["state"])[~touched], c["state64"][~touched])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("seqs,H", [(1, 1), (1, 16), (7, 3), (33, 5)])
def test_step_single_tokens(tpc, d, dt, seqs, H):
    import torch
    rng = np.random.default_rng(d + seqs + H)
    c = step_case(rng, seqs, H, d, torch.float32 if dt == "f32" else torch.bfloat16)
    check_step(tpc, c)


@pytest.mark.parametrize("d,dt,out", [(128, "bf16", "f32"), (64, "f32", "bf16"), (32, "bf16", "bf16"), (128, "f32", "f32")])
@pytest.mark.parametrize("fork", [False, True])
def test_step_runs(tpc, d, dt, out, fork):
    """Ragged runs (none, one and many rows), rows behind the last sequence, padding entries, branches."""
    import torch
    rng = np.random.default_rng(d + 100 * fork)
    tt = {"f32": torch.float32, "bf16": torch.bfloat16}
    c = step_case(rng, 6, 3, d, tt[dt], m=[3, 0, 1, 9, 0, 2], extra_rows=2, fork=fork)
    c["src"][2] = -1
    check_step(tpc, c, out_dtype=tt[out])


def test_step_empty_batches(tpc):
    import torch
    rng = np.random.default_rng(9)
    c = step_case(rng, 3, 2, 64, torch.float32, m=[0, 0, 0], fork=True)  # branches without a token: states are copied
    check_step(tpc, c)
    c = step_case(rng, 0, 2, 64, torch.float32, m=np.zeros(0, int), slots=2)
    check_step(tpc, c)


def test_step_gates_of_any_size(tpc):
    """Gates down to -infinity: the channel's state is dropped, and nothing becomes NaN."""
    import torch
    rng = np.random.default_rng(10)
    c = step_case(rng, 4, 2, 128, torch.float32, m=[2, 1, 3, 1])
    g = c["g64"].copy()
    g[:, :, ::3] = -np.inf
    g[:, :, 1::3] = -200.0
    c["g"], c["g64"] = dev(g, torch.float32), g
    check_step(tpc, c)


def test_step_bad_slots(tpc):
    """Slots outside the cache, and a slot that two sequences share in a way that races, set the status."""
    import torch
    rng = np.random.default_rng(11)
    for src, dst, start in ([[0, 9, 1], None, None], [[0, 1, 2], [3, 4, -1], None], [[0, 1, 2], [3, 4, 9], None],
                            [[0, 1, 0], None, None], [[0, 1, 2], [3, 4, 3], None], [[0, 1, 2], [3, 0, 4], None],
                            [[0, 1, 2], None, [0, 2, 1, 3]], [[0, 1, 2], None, [0, 1, 2, 4]], [[0, 1, 2], None, [-1, 1, 2, 3]]):
        c = step_case(rng, 3, 2, 64, torch.float32, slots=9)
        before = c["state"].clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tpc.tpc_kda_step(c["state"], dev(np.array(src, np.int32)), c["q"], c["k"], c["v"], c["g"], c["beta"],
                         dst=None if dst is None else dev(np.array(dst, np.int32)),
                         row_start=None if start is None else dev(np.array(start, np.int32)), status=status)
        assert status.item() == 7, (src, dst, start)
        touched = [s for s in (src if dst is None else dst) if 0 <= s < 9]
        rest = [i for i in range(9) if i not in touched]
        assert torch.equal(c["state"][rest], before[rest])
    # several readers of one slot, none of them writing it, are branches and not a race
    c = step_case(rng, 3, 2, 64, torch.float32, slots=9)
    c["src"], c["dst"] = np.array([2, 2, 5], np.int32), np.array([0, 1, 5], np.int32)
    check_step(tpc, c)


def test_step_continues_the_tree_forward(tpc):
    """A prompt through the tree-packed forward, then its final state token by token: the outputs are those of
    the forward over the whole trajectory.  Both are fp32 evaluations of one recurrence; the bound is the
    forward's own (1e-5 of the RMS) and the step's."""
    import torch
    rng = np.random.default_rng(12)
    T, P, H, d = 90, 71, 2, 64
    x = {k: dev(rng.normal(size=(T, H, d)), torch.float32) for k in "qkv"}
    x["k"] /= x["k"].norm(dim=-1, keepdim=True)
    x["g"] = -0.1 * torch.nn.functional.softplus(dev(rng.normal(size=(T, H, d)), torch.float32))
    x["beta"] = torch.sigmoid(dev(rng.normal(size=(T, H)), torch.float32))
    full = tpc.Plan([-1], [T], 32).upload()
    o_ref, fin_ref, _ = tpc.tpc_kda_forward(full, *(x[k] for k in ("q", "k", "v", "g", "beta")))
    head = tpc.Plan([-1], [P], 32).upload()
    o, state, _ = tpc.tpc_kda_forward(head, *(x[k][:P].contiguous() for k in ("q", "k", "v", "g", "beta")))
    src = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [o]
    for t in range(P, T - 8):
        outs.append(tpc.tpc_kda_step(state, src, *(x[k][t:t + 1] for k in ("q", "k", "v", "g", "beta"))))
    outs.append(tpc.tpc_kda_step(state, src, *(x[k][T - 8:] for k in ("q", "k", "v", "g", "beta")),
                                 row_start=dev(np.array([0, 8], np.int32))))
    rms = lambda t: float(t.double().pow(2).mean().sqrt())
    assert float((torch.cat(outs) - o_ref).abs().max()) <= 3e-5 * rms(o_ref)
    assert float((state - fin_ref).abs().max()) <= 3e-5 * rms(fin_ref)


# ------------------------------------------------------------------------------------ paged cache
def batch(rng, kv, page, n_pages=None, shared=0):
    """A scattered block table for the given lengths; the first `shared` pages of all sequences are one."""
    per = max(1, max(-(-int(x) // page) for x in kv))
    need = len(kv) * per + 2
    n_pages = n_pages or need
    table = rng.permutation(need)[:len(kv) * per].reshape(len(kv), per).astype(np.int32)
    table[:, :shared] = table[0, :shared]
    return table, n_pages


@pytest.mark.parametrize("page", [16, 32, 64, 192])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append(tpc, page, dt):
    import torch
    rng = np.random.default_rng(page)
    m, kv = [3, 0, 1, 70, 2, 5], [3, 9, 40, 200, 0, 2]  # a fresh, an idle, a padding entry, one longer than its length
    n = sum(m) + 3
    table, n_pages = batch(rng, kv, page)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    cache, c64 = rounded(rng, n_pages, page, 576, dtype=torch.bfloat16)
    proj, p64 = rounded(rng, n, 3 * 192 + 576, dtype=dtype)  # slices of a projection
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tpc.tpc_latent_append(cache, dev(table), dev(np.array(kv, np.int32)), proj[:, 576:1088], proj[:, 1088:],
                          row_start=dev(starts(m)), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref = od.append(c64, table, kv, p64[:, 576:1088], p64[:, 1088:], starts(m))
    x = host(cache)
    lat = ref[..., :512] if dt == "bf16" else host(dev(ref[..., :512], torch.float32).to(torch.bfloat16))
    assert np.array_equal(x[..., :512], lat)
    # a rotated value: two products and a sum of fp32 with cos, sin within 2^-21, then one rounding
    tol = UBF * np.abs(ref[..., 512:]) + 2.0 ** -19 * np.abs(p64[:, 1088:]).max()
    within(x[..., 512:], ref[..., 512:], tol, "rotary key")


def test_append_far_positions_and_single_tokens(tpc):
    """One row a sequence without row_start, up to positions whose angles exceed fp32's exact integers."""
    import torch
    rng = np.random.default_rng(5)
    kv = np.array([1, 64, 65, 0, 2_000_003, 1_048_577], np.int32)
    page = 2 ** 20
    table = np.arange(12, dtype=np.int32).reshape(6, 2) % 6
    table = np.array([[0, 5], [1, 5], [2, 5], [3, 5], [5, 4], [5, 3]], np.int32)
    cache = torch.zeros(6, page, 576, dtype=torch.bfloat16, device="cuda")
    c, c64 = rounded(rng, 6, 512, dtype=torch.bfloat16)
    kr, k64 = rounded(rng, 6, 64, dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(tpc.TpcError):  # one dtype for both
        tpc.tpc_latent_append(cache, dev(table), dev(kv), c, kr)
    kr = kr.to(torch.bfloat16)
    k64 = host(kr)
    tpc.tpc_latent_append(cache, dev(table), dev(kv), c, kr, status=status)
    assert status.item() == 0
    written = 0
    for b in range(6):
        p = int(kv[b]) - 1
        if p < 0:
            continue
        row = host(cache[table[b, p // page], p % page])
        assert np.array_equal(row[:512], c64[b])
        ref = od.rotate(k64[b], p)
        within(row[512:], ref, UBF * np.abs(ref) + 2.0 ** -19 * np.abs(k64[b]).max(), b)
        written += 1
    assert int((cache != 0).any(-1).sum()) == written  # and nothing else


def test_append_bad_tables(tpc):
    import torch
    rng = np.random.default_rng(6)
    c, _ = rounded(rng, 3, 512, dtype=torch.bfloat16)
    kr, _ = rounded(rng, 3, 64, dtype=torch.bfloat16)

    def status_of(table, kv, start=None):
        cache = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tpc.tpc_latent_append(cache, dev(np.array(table, np.int32)), dev(np.array(kv, np.int32)), c, kr,
                              row_start=None if start is None else dev(np.array(start, np.int32)), status=status)
        return status.item(), int((cache != 0).any(-1).sum())

    assert status_of([[0, 1], [2, 1], [3, 1]], [16, 3, 1]) == (0, 3)
    assert status_of([[0, 1], [4, 1], [3, 1]], [16, 3, 1]) == (7, 2)     # a page outside the cache
    assert status_of([[0, 1], [-1, 1], [3, 1]], [16, 3, 1]) == (7, 2)
    assert status_of([[0, 1], [2, 1], [3, 1]], [33, 3, 1]) == (7, 2)     # a position outside the table
    assert status_of([[0, 1], [2, 1], [0, 1]], [16, 3, 1])[0] == 7       # two sequences write one page
    assert status_of([[0, 1], [2, 1], [0, 1]], [16, 18, 18])[0] == 7
    assert status_of([[0, 1], [0, 2], [0, 3]], [17, 17, 17]) == (0, 3)   # a shared full page that no one writes
    assert status_of([[0, 0]], [17], [0, 3])[0] == 7                     # one page twice in the written range


# ------------------------------------------------------------------------------------ absorb, expand
@pytest.mark.parametrize("H,m,kv", [(1, [1], [1]), (16, [1], [70000]), (5, [1] * 9, list(range(9))), (3, [4, 0, 130, 1], [4, 0, 5000, 0]),
                                    (16, [127, 2, 129], [127, 9, 200000]), (128, [2, 1], [2, 7])])
def test_absorb(tpc, H, m, kv):
    import torch
    rng = np.random.default_rng(H + len(m))
    ragged = any(x != 1 for x in m)
    n = sum(m) + (2 if ragged else 0)
    wide, w64 = rounded(rng, n, H * 192 + 64, dtype=torch.bfloat16)
    q = wide[:, :H * 192].unflatten(1, (H, 192))
    w_b, wb64 = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
    qa = torch.full((n, H, 576), -7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = starts(m) if ragged else None
    got = tpc.tpc_latent_absorb(q, w_b, dev(np.array(kv, np.int32)), row_start=None if start is None else dev(start), qa=qa,
                                status=status)
    torch.cuda.synchronize()
    assert got is qa and status.item() == 0
    ref, mag = od.absorb(w64[:, :H * 192].reshape(n, H, 192), wb64, kv, start)
    own = ~np.isnan(ref)
    x = host(qa)
    assert (x[~own] == -7.0).all()
    tol = UBF * np.abs(ref) + np.where(np.arange(576) < 512, 140 * U32, 2.0 ** -19) * mag
    within(x[own], ref[own], tol[own], "qa")


@pytest.mark.parametrize("n,H", [(1, 1), (1, 16), (9, 5), (127, 3), (130, 16), (300, 2), (2, 128)])
def test_expand(tpc, n, H):
    import torch
    rng = np.random.default_rng(n + H)
    o, o64 = rounded(rng, n, H, 512, dtype=torch.bfloat16)
    w_b, wb64 = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tpc.tpc_latent_expand(o, w_b, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref, mag = od.expand(o64, wb64)
    within(host(out), ref, UBF * np.abs(ref) + 520 * U32 * mag, "out")


# ------------------------------------------------------------------------------------ attention
def check_attention(tpc, rng, H, m, kv, page, shared=0, poison=True, extra=0, scale=SCALE, s=1.0, scratch=None, table=None):
    import torch
    ragged = extra or any(x != 1 for x in m)
    n = sum(m) + extra
    table, n_pages = batch(rng, kv, page, shared=shared) if table is None else (table, int(table.max()) + 1)
    cache, c64 = rounded(rng, n_pages, page, 576, dtype=torch.bfloat16)
    if poison:  # whatever lies past the sequences' tokens is never used
        used = np.zeros((n_pages, page), bool)
        for b, L in enumerate(kv):
            for j in range(0, L, page):
                used[table[b, j // page], :min(page, L - j)] = True
        cache[dev(~used)] = float("nan")
        idle = np.argwhere(~used)
        for i, (p, r) in enumerate(idle[::3]):
            cache[int(p), int(r)] = float("inf") if i < 50 else float("nan")
            if i > 60:
                break
    qa, q64 = rounded(rng, n, H, 576, dtype=torch.bfloat16, s=s)
    o = torch.full((n, H, 512), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = starts(m) if ragged else None
    args = (qa, cache, dev(table), dev(np.array(kv, np.int32)), scale)
    kw = dict(row_start=None if start is None else dev(start), scratch=scratch)
    tpc.tpc_latent_attn(*args, o=o, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref, lref, oa, sa = od.attention(q64, np.nan_to_num(c64), table, kv, scale, start)
    own = ~np.isnan(lref)
    x, l = host(o), host(lse)
    assert (x[~own] == -7.0).all() and (l[~own] == -7.0).all()
    ds = 640 * U32 * sa
    L = max(list(kv) + [1])
    tol = UBF * np.abs(ref) + (UBF + 2 * ds[..., None] + 2.0 ** -14 + L * U32) * oa
    within(x[own], ref[own], tol[own], "o")
    ltol = ds + 2.0 ** -18 + L * U32 + 4 * U32 * np.abs(np.where(np.isfinite(lref), lref, 0))
    within(l[own], lref[own], ltol[own], "lse")
    again = tpc.tpc_latent_attn(*args, **kw)
    assert torch.equal(again[0][dev(own[:, 0])], o[dev(own[:, 0])]) and torch.equal(again[1][dev(own[:, 0])], lse[dev(own[:, 0])])


@pytest.mark.parametrize("kv", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 1000, 4097])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_lengths(tpc, kv, page):
    check_attention(tpc, np.random.default_rng(kv + page), 16, [1], [kv], page)


@pytest.mark.parametrize("H", [1, 2, 5, 8, 16, 17, 24, 32, 33, 64, 100, 128])
def test_attention_heads(tpc, H):
    check_attention(tpc, np.random.default_rng(H), H, [1, 1, 1], [130, 0, 77], 32)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 192])
@pytest.mark.parametrize("H", [3, 16])
def test_attention_runs(tpc, H, page):
    """Ragged runs with causal rows: whole prompts, one more token, none, padding entries, rows behind the end."""
    rng = np.random.default_rng(page + H)
    check_attention(tpc, rng, H, [7, 0, 1, 70, 3, 2, 1], [300, 20, 64, 70, 0, 1, 1025], page, extra=3)


def test_attention_batches(tpc):
    """Many sequences (more than a block has threads), shared prefixes, all lengths mixed."""
    rng = np.random.default_rng(21)
    kv = [int(x) for x in rng.integers(0, 260, 400)]
    check_attention(tpc, rng, 4, [1] * 400, kv, 32)
    kv = [int(x) for x in rng.integers(129, 900, 9)]
    check_attention(tpc, rng, 16, [1] * 9, kv, 64, shared=2)
    check_attention(tpc, rng, 16, [int(x) for x in rng.integers(0, 5, 150)], [int(x) for x in rng.integers(5, 600, 150)], 16)


def test_attention_of_short_tables(tpc):
    """Tables of at most 128 tokens (one tile a context, no joining) and just above, many and few sequences."""
    rng = np.random.default_rng(25)
    for page, top in ((16, 128), (32, 129), (64, 100), (128, 128), (192, 150)):
        kv = [int(x) for x in rng.integers(0, top + 1, 30)] + [top]
        check_attention(tpc, rng, 16, [1] * 31, kv, page)
        check_attention(tpc, rng, 5, [0, 9, 3], [4, top, 17], page)
        check_attention(tpc, rng, 40, [1], [top], page)


@pytest.mark.parametrize("s", [0.01, 8.0, 60.0])
def test_attention_score_ranges(tpc, s):
    """Nearly uniform and nearly one-hot softmaxes (scores of hundreds), whose maximum moves along the row."""
    check_attention(tpc, np.random.default_rng(int(s * 100)), 16, [1, 3], [2000, 900], 64, s=s)


def test_attention_rising_and_falling_scores(tpc):
    """Scores that rise, then fall along the context: the running maximum moves at every tile, or never."""
    import torch
    rng = np.random.default_rng(22)
    for sign in (1, -1):
        L, H, page = 700, 16, 64
        qa = torch.zeros(1, H, 576, dtype=torch.bfloat16, device="cuda")
        qa[:, :, 0] = 8.0
        cache, _ = rounded(rng, 11, page, 576, dtype=torch.bfloat16)
        ramp = torch.arange(704, device="cuda").view(11, page).float() * (sign * 0.25)
        cache[:, :, 0] = ramp.to(torch.bfloat16)
        table = np.arange(11, dtype=np.int32)[None]
        o, lse = tpc.tpc_latent_attn(qa, cache, dev(table), dev(np.array([L], np.int32)), 1.0)
        ref, lref, oa, sa = od.attention(host(qa), host(cache), table, [L], 1.0)
        tol = UBF * np.abs(ref) + (UBF + 2.0 ** -14 + 1280 * U32 * sa[..., None]) * oa
        within(host(o), ref, tol, "o")
        within(host(lse), lref, 640 * U32 * sa + 2.0 ** -18 + 4 * U32 * np.abs(lref), "lse")


def test_attention_bad_tables(tpc):
    """Entries outside the cache and lengths outside the table set the status; the other sequences are right."""
    import torch
    rng = np.random.default_rng(23)
    cache, c64 = rounded(rng, 6, 16, 576, dtype=torch.bfloat16)
    qa, q64 = rounded(rng, 2, 4, 576, dtype=torch.bfloat16)
    for table, kv in ([[[0, 1], [2, 6]], [20, 20]], [[[0, 1], [-5, 2]], [20, 3]], [[[0, 1], [2, 3]], [20, 33]]):
        table = np.array(table, np.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = tpc.tpc_latent_attn(qa, cache, dev(table), dev(np.array(kv, np.int32)), SCALE, status=status)
        assert status.item() == 7, (table, kv)
        ref, lref, oa, _ = od.attention(q64[:1], c64, table[:1], kv[:1], SCALE)
        within(host(o)[:1], ref, UBF * np.abs(ref) + (UBF + 2.0 ** -10) * oa, "o")
    # an entry that no token reaches may hold anything
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tpc.tpc_latent_attn(qa, cache, dev(np.array([[0, 99], [1, -1]], np.int32)), dev(np.array([16, 5], np.int32)), SCALE, status=status)
    assert status.item() == 0


def test_bad_row_starts(tpc):
    """Row tables that decrease or leave the rows: reported by the step and the attention, followed by no call
    (what lies around the tensors keeps its values)."""
    import torch
    rng = np.random.default_rng(24)
    H, big = 2, 2 ** 31 - 1
    i32 = lambda a: dev(np.array(a, np.int32))
    for start in ([0, 2, 1, 3], [-4, 1, 2, 3], [0, 1, 2, 9], [big, 0, 1, 3], [0, -big, big, 3], [3, 2, 1, 0]):
        guard = torch.full((9, H, 576), -7.0, dtype=torch.bfloat16, device="cuda")
        qa, w_b, cache = (rounded(rng, *s, dtype=torch.bfloat16)[0] for s in ((3, H, 576), (512, 512), (6, 16, 576)))
        table, kv = i32(rng.permutation(6).reshape(3, 2)), i32([20, 5, big])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qo = guard.clone()
        tpc.tpc_latent_absorb(qa[:, :, :192].contiguous(), w_b, kv, row_start=i32(start), qa=qo[3:6], status=status)
        c, kr = rounded(rng, 3, 512, dtype=torch.bfloat16)[0], rounded(rng, 3, 64, dtype=torch.bfloat16)[0]
        pool = guard.new_full((18, 16, 576), -7.0)
        tpc.tpc_latent_append(pool[6:12], table, kv, c, kr, row_start=i32(start), status=status)
        ao, al = guard.new_full((9, H, 512), -7.0), torch.full((9, H), -7.0, device="cuda")
        status.zero_()
        tpc.tpc_latent_attn(qa, cache, table, kv, SCALE, row_start=i32(start), o=ao[3:6], lse=al[3:6], status=status)
        assert status.item() == 7, start
        for t in (qo, ao, al):
            assert bool((t[:3] == -7).all()) and bool((t[6:] == -7).all()), start
        assert bool((pool[:6] == -7).all()) and bool((pool[12:] == -7).all()), start
        x, st = rounded(rng, 3, H, 64, dtype=torch.float32)[0], rounded(rng, 9, H, 64, 64, dtype=torch.float32)[0]
        keep, so = st.clone(), torch.full((9, H, 64), -7.0, device="cuda")
        status.zero_()
        tpc.tpc_kda_step(st[3:6], i32([0, 1, 2]), x, x, x, -x.abs(), x[:, :, 0].contiguous(), row_start=i32(start), o=so[3:6], status=status)
        assert status.item() == 7, start
        assert torch.equal(st[:3], keep[:3]) and torch.equal(st[6:], keep[6:])
        assert bool((so[:3] == -7).all()) and bool((so[6:] == -7).all()), start


# ------------------------------------------------------------------------------------ together
def test_generation_matches_the_expanded_attention(tpc):
    """A prompt and then single tokens through append, absorb, attention and expand equal the expanded causal
    attention over the whole sequence.  Each of the three roundings on the way (absorbed queries, attention
    outputs, head outputs) is off by half a step; with scores of unit size a query rounding moves a weight by
    at most 2^-8 times the sum of |q k| scale, so 6 half-steps of the summed magnitudes bound the whole."""
    import torch
    rng = np.random.default_rng(30)
    T, P, H, page = 150, 129, 16, 32
    q, q64 = rounded(rng, T, H, 192, dtype=torch.bfloat16, s=0.5)
    c, c64 = rounded(rng, T, 512, dtype=torch.bfloat16)
    kr, k64 = rounded(rng, T, 64, dtype=torch.bfloat16)
    w_b, w64 = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.02)
    cache = torch.full((8, page, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = dev(np.array([[6, 1, 3, 0, 5]], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scratch = tpc.latent_attn_scratch(H)
    outs = []
    for a, b in [(0, P)] + [(t, t + 1) for t in range(P, T)]:
        kv = dev(np.array([b], np.int32))
        start = dev(np.array([0, b - a], np.int32))
        tpc.tpc_latent_append(cache, table, kv, c[a:b], kr[a:b], row_start=start, status=status)
        qa = tpc.tpc_latent_absorb(q[a:b], w_b, kv, row_start=start, status=status)
        o, _ = tpc.tpc_latent_attn(qa, cache, table, kv, SCALE, row_start=start, scratch=scratch, status=status)
        outs.append(tpc.tpc_latent_expand(o, w_b, status=status))
    assert status.item() == 0
    ref = od.expanded_attention(q64, c64, k64, w64, SCALE)
    x = host(torch.cat(outs))
    v = np.einsum("tl,hil->thi", np.abs(c64), np.abs(w64[H * 128:]).reshape(H, 128, 512))
    mag = np.cumsum(v, 0) / np.arange(1, T + 1)[:, None, None]
    # weights of unit-size scores are within e^2 of uniform, so mag e^2 bounds the weighted sums of magnitudes
    within(x, ref, 6 * UBF * mag * np.e ** 2, "generation")
    rms = np.sqrt(np.mean((x - ref) ** 2) / np.mean(ref ** 2))
    assert rms < 4 * UBF, rms  # and the errors are independent roundings, not a shift


def test_capture_and_replay(tpc):
    """One captured step of both layers, replayed with new rows, lengths and slots in the same buffers."""
    import torch
    rng = np.random.default_rng(31)
    B, H, page = 5, 4, 16
    w_b, _ = rounded(rng, 2 * H * 128, 512, dtype=torch.bfloat16, s=0.05)
    table = dev(rng.permutation(20).reshape(B, 4).astype(np.int32))
    bf = torch.bfloat16
    fresh = lambda: dict(q=rounded(rng, B, H, 192, dtype=bf)[0], c=rounded(rng, B, 512, dtype=bf)[0], kr=rounded(rng, B, 64, dtype=bf)[0],
                         kv=dev(rng.integers(0, 64, B).astype(np.int32)), src=dev(rng.permutation(B).astype(np.int32)),
                         x=rounded(rng, B, H, 64, dtype=bf)[0], g=dev(-np.abs(rng.normal(size=(B, H, 64))), bf),
                         beta=dev(rng.uniform(size=(B, H)), bf))
    cache0, _ = rounded(rng, 20, page, 576, dtype=bf)
    state0, _ = rounded(rng, B, H, 64, 64, dtype=torch.float32)

    def step(b, cache, state, scratch):
        tpc.tpc_latent_append(cache, table, b["kv"], b["c"], b["kr"])
        qa = tpc.tpc_latent_absorb(b["q"], w_b, b["kv"])
        o, lse = tpc.tpc_latent_attn(qa, cache, table, b["kv"], SCALE, scratch=scratch)
        return tpc.tpc_latent_expand(o, w_b), lse, tpc.tpc_kda_step(state, b["src"], b["x"], b["x"], b["x"], b["g"], b["beta"])

    buf, scratch = fresh(), tpc.latent_attn_scratch(H)
    cache, state = cache0.clone(), state0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buf, cache0.clone(), state0.clone(), scratch)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(buf, cache, state, scratch)
    ref_cache, ref_state = cache0.clone(), state0.clone()
    for _ in range(3):
        new = fresh()
        for k in buf:
            buf[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        ref = step(new, ref_cache, ref_state, tpc.latent_attn_scratch(H))
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        assert torch.equal(cache, ref_cache) and torch.equal(state, ref_state)


def test_two_streams_with_scratch_of_their_own(tpc):
    """Two calls at once, each on its stream (given as an argument), equal the same calls alone."""
    import torch
    rng = np.random.default_rng(32)
    H, kv, page = 16, [3000, 1777, 64], 64
    table, n_pages = batch(rng, kv, page)
    cache, _ = rounded(rng, n_pages, page, 576, dtype=torch.bfloat16)
    qs = [rounded(rng, 3, H, 576, dtype=torch.bfloat16)[0] for _ in range(2)]
    tb, kvd = dev(table), dev(np.array(kv, np.int32))
    alone = [tpc.tpc_latent_attn(q, cache, tb, kvd, SCALE) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [tpc.tpc_latent_attn(q, cache, tb, kvd, SCALE, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_wrappers_refuse(tpc):
    import torch
    bf = torch.bfloat16
    z = lambda *s, t=bf: torch.zeros(*s, dtype=t, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    before = tpc.tpc_launch_count()
    x, st = z(2, 3, 64), z(4, 3, 64, 64, t=torch.float32)
    ok = dict(state=st, src=i(2), q=x, k=x, v=x, g=x, beta=z(2, 3))
    for name, bad in (("state", z(4, 3, 64, 64)), ("state", z(4, 2, 64, 64, t=torch.float32)), ("src", i(3)), ("src", i(2).long()),
                      ("k", x.float()), ("q", z(2, 3, 64, t=torch.float16)), ("v", z(2, 3, 32)), ("beta", z(2, 3, 1)),
                      ("g", z(2, 64, 3).transpose(1, 2)), ("beta", z(2, 3).cpu()), ("dst", i(1)), ("row_start", i(2)),
                      ("o", z(2, 3, 32)), ("status", i(0)), ("out_dtype", torch.float16)):
        with pytest.raises(tpc.TpcError):
            tpc.tpc_kda_step(**{**ok, name: bad})
    ok = dict(cache=z(4, 16, 576), block_table=i(2, 2), kv_len=i(2), c=z(2, 512), kr=z(2, 64))
    for name, bad in (("cache", z(4, 16, 512)), ("cache", z(4, 24, 576)), ("cache", z(64, 576)), ("block_table", i(3, 2)),
                      ("block_table", i(2, 2).long()), ("kv_len", i(3)), ("c", z(2, 576)), ("c", z(512, 2).T), ("kr", z(3, 64)),
                      ("kr", z(2, 64, t=torch.float32)), ("c", z(2, 513)[:, 1:]), ("row_start", i(2))):
        with pytest.raises(tpc.TpcError):
            tpc.tpc_latent_append(**{**ok, name: bad})
    ok = dict(q=z(2, 3, 192), w_b=z(768, 512), kv_len=i(2))
    for name, bad in (("q", z(2, 3, 128)), ("q", z(3, 2, 192).transpose(0, 1)), ("w_b", z(512, 512)), ("kv_len", i(1)), ("qa", z(2, 3, 512)),
                      ("q", z(2, 3, 192, t=torch.float32))):
        with pytest.raises(tpc.TpcError):
            tpc.tpc_latent_absorb(**{**ok, name: bad})
    ok = dict(qa=z(2, 3, 576), cache=z(4, 16, 576), block_table=i(2, 2), kv_len=i(2), scale=0.1)
    for name, bad in (("qa", z(2, 3, 512)), ("qa", z(2, 129, 576)), ("cache", z(4, 16, 576, t=torch.float32)), ("kv_len", i(3)),
                      ("o", z(2, 3, 512, t=torch.float32)), ("lse", z(2, 3)), ("scratch", z(64, t=torch.uint8)), ("block_table", i(2))):
        with pytest.raises(tpc.TpcError):
            tpc.tpc_latent_attn(**{**ok, name: bad})
    for o, w in ((z(2, 3, 128), z(768, 512)), (z(2, 3, 512), z(384, 512)), (z(2, 129, 512), z(256 * 129, 512))):
        with pytest.raises(tpc.TpcError):
            tpc.tpc_latent_expand(o, w)
    assert tpc.tpc_launch_count() == before


def test_sampled_branches_match_the_layer_group(tpc):
    """One KDA and one latent-attention layer of the hybrid group (2048 wide, 16 heads): a prompt, then two branches
    sampled token by token from its state and its shared pages, against tpc_group_forward over the whole tree.
    The KDA layer's rows are fp32 on both sides (the group is held to 2e-3 of the RMS, so are its states here).
    The attention's part of y goes through eight bf16 roundings (q, c, kr, qa, the weights of the softmax, o, the
    head outputs, and the scores they move), each off by at most half a step: 8 2^-8 of its RMS."""
    import torch
    D, H, hd, page, P = 2048, 16, 128, 16, 70
    branch = [5, 9]
    g = torch.Generator(device="cuda").manual_seed(40)
    rnd = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale
    W = {"kda": [(rnd(4 * D + H, D, scale=0.02).bfloat16(), rnd(D, D, scale=0.02).bfloat16())],
         "mla": (rnd(H * 192 + 576, D, scale=0.02).bfloat16(), rnd(2 * D, 512, scale=0.02).bfloat16(), rnd(D, D, scale=0.02).bfloat16())}
    rows = {0: rnd(P, D), 1: rnd(branch[0], D), 2: rnd(branch[1], D)}
    tree = tpc.Plan([-1, 0, 0], [P] + branch, 64).upload()
    at = tree.tables()["row_offset"]
    x = torch.empty(P + sum(branch), D, device="cuda")
    for v, r in rows.items():
        x[at[v]:at[v] + len(r)] = r
    ws = tpc.group_workspace(tree, 1)
    y_ref, h_ref = tpc.tpc_group_forward(tree, W, x, ws)
    assert tpc.tpc_group_status(tree, ws, 1) == 0

    norm = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6)
    mul = lambda t, w: t @ w.float().T

    def kda_inputs(t):
        p = mul(norm(t), W["kda"][0][0])
        q, k, v, gt = (p[:, i * D:(i + 1) * D].reshape(-1, H, hd) for i in range(4))
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
        return [z.contiguous() for z in (q, k, v, -0.1 * torch.nn.functional.softplus(gt), torch.sigmoid(p[:, 4 * D:]))]

    # the prompt: its KDA state by the chunkwise forward, its latents from the group's KDA output
    prompt = tpc.Plan([-1], [P], 64).upload()
    state = torch.zeros(3, H, hd, hd, device="cuda")
    o, fin, _ = tpc.tpc_kda_forward(prompt, *kda_inputs(rows[0]), split=True)
    state[0] = fin[0]
    h0 = h_ref[0][at[0]:at[0] + P]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = torch.full((16, page, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    shared, last = [3, 9, 1, 12], 7  # 64 tokens in full pages, six in a page of their own
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    proj = mul(norm(h0), W["mla"][0])
    tpc.tpc_latent_append(cache, i32(*shared, last)[None], i32(P), proj[:, H * 192:H * 192 + 512], proj[:, H * 192 + 512:],
                          row_start=i32(0, P), status=status)
    cache[4], cache[10] = cache[last], cache[last]  # a branch writes into a copy of the partial page
    table = torch.stack([i32(*shared, 4), i32(*shared, 10)])
    scratch = tpc.latent_attn_scratch(H)
    got_y, got_h, kept = {1: [], 2: []}, {1: [], 2: []}, cache[shared].clone()
    for t in range(max(branch)):
        live = [b for b in range(2) if t < branch[b]]
        xt = torch.stack([rows[1 + b][t] for b in live])
        dst = i32(*(1 + b for b in live))
        src = i32(*([0] * len(live))) if t == 0 else dst  # both branches start from the prompt's state
        o = tpc.tpc_kda_step(state, src, *kda_inputs(xt), dst=dst, status=status)
        ht = xt + mul(o.reshape(-1, D), W["kda"][0][1])
        proj = mul(norm(ht), W["mla"][0])
        kv, tab = i32(*(P + t + 1 for _ in live)), table[live].contiguous()
        tpc.tpc_latent_append(cache, tab, kv, proj[:, H * 192:H * 192 + 512], proj[:, H * 192 + 512:], status=status)
        qa = tpc.tpc_latent_absorb(proj[:, :H * 192].bfloat16().view(-1, H, 192), W["mla"][1], kv, status=status)
        o, _ = tpc.tpc_latent_attn(qa, cache, tab, kv, SCALE, scratch=scratch, status=status)
        o = tpc.tpc_latent_expand(o, W["mla"][1], status=status)
        yt = ht + mul(o.float().reshape(-1, D), W["mla"][2])
        for i, b in enumerate(live):
            got_h[1 + b].append(ht[i])
            got_y[1 + b].append(yt[i])
    assert status.item() == 0 and torch.equal(cache[shared], kept)
    rms = lambda t: float(t.double().pow(2).mean().sqrt())
    for v in (1, 2):
        ref_h, ref_y = (z[at[v]:at[v] + branch[v - 1]] for z in (h_ref[0], y_ref))
        h, y = torch.stack(got_h[v]), torch.stack(got_y[v])
        assert float((h - ref_h).abs().max()) <= 4e-3 * rms(ref_h)
        err = rms((y - h) - (ref_y - ref_h)) / rms(ref_y - ref_h)
        assert err <= 8 * UBF, err


def test_offsets_past_32_bits(tpc):
    """Caches of more than 2^31 elements: slots and pages at their far end."""
    import torch
    rng = np.random.default_rng(41)
    H, d, slots = 16, 128, 8300  # 2.18e9 fp32 state elements
    c = step_case(rng, 2, H, d, torch.bfloat16)
    state = torch.empty(slots, H, d, d, device="cuda")
    far = np.array([slots - 1, slots - 3], np.int32)
    state[dev(far).long()] = c["state"][:2]
    c["src"], small = np.array([0, 1], np.int32), c["state"][:2].clone()
    args = (c["q"], c["k"], c["v"], c["g"], c["beta"])
    want = tpc.tpc_kda_step(small, dev(c["src"]), *args)
    got = tpc.tpc_kda_step(state, dev(far), *args)
    assert torch.equal(got, want) and torch.equal(state[dev(far).long()], small)
    del state
    pages, page = 60000, 64  # 2.2e9 bf16 cache elements
    cache = torch.empty(pages, page, 576, dtype=torch.bfloat16, device="cuda")
    near, _ = rounded(rng, 6, page, 576, dtype=torch.bfloat16)
    order = torch.tensor([pages - 1, pages - 5, 58255, pages - 2, pages - 7, 58254], device="cuda")  # 2^31 / (64 * 576) = 58254.2
    cache[order] = near
    kv = dev(np.array([130, 177], np.int32))
    x, _ = rounded(rng, 2, 576, dtype=torch.bfloat16)
    qa, _ = rounded(rng, 2, 16, 576, dtype=torch.bfloat16)
    t_near, t_far = dev(np.arange(6, dtype=np.int32).reshape(2, 3)), order.int().view(2, 3)
    res = []
    for ch, tb in ((near, t_near), (cache, t_far)):
        tpc.tpc_latent_append(ch, tb, kv, x[:, :512], x[:, 512:])
        res.append(tpc.tpc_latent_attn(qa, ch, tb, kv, SCALE))
    assert torch.equal(cache[order], near)
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_attention_of_idle_and_long_sequences(tpc):
    """Thousands of sequences of which few have a row, and one long context among empty ones."""
    rng = np.random.default_rng(42)
    m, kv = [0] * 3000, [0] * 3000
    table = np.zeros((3000, 63), np.int32)  # idle sequences' entries are page 0
    for i, (b, (rows, length)) in enumerate({7: (1, 33), 1500: (5, 4000), 2999: (2, 700)}.items()):
        m[b], kv[b], table[b] = rows, length, 1 + 63 * i + rng.permutation(63)
    check_attention(tpc, rng, 8, m, kv, 64, poison=False, table=table)
    table = np.zeros((20, 282), np.int32)
    table[10] = 1 + rng.permutation(282)
    check_attention(tpc, rng, 16, [1] * 20, [0] * 10 + [9000] + [0] * 9, 32, poison=False, table=table)
