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
