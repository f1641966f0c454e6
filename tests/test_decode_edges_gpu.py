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
