"""Token-by-token generation, host side (no GPU): the calls refuse bad arguments before any launch."""
import ctypes as C

import numpy as np
import pytest

from oracle import decode as od


@pytest.fixture(scope="module")
def tpc():
    from tree_packed_chunkwise_b200 import build
    build.build()
    import tree_packed_chunkwise_b200 as t
    t.lib()
    return t


A = 1 << 20  # an aligned address that no call may follow


def rows(tpc, n=4, seqs=4, start=None, kv=A):
    return C.byref(tpc.Rows(n, seqs, start, kv))


def cache(tpc, data=A, n_pages=8, page=64, table=A, max_pages=2):
    return C.byref(tpc.LatentCache(data, n_pages, page, table, max_pages))


def step(tpc, rws=None, H=2, d=128, dv=None, din=1, dout=1, **io):
    f = dict(q=A, k=A, v=A, g=A, beta=A, state=A, n_slots=8, src=A, dst=None, o=A)
    f.update(io)
    sh = tpc.KdaShape(H, d, d if dv is None else dv, din, dout)
    return tpc.lib().tpc_kda_step(C.byref(sh), rws or rows(tpc), C.byref(tpc.KdaStepIO(**f)), None, None)


NULL, SHAPE, UNSUP, WS = 4, 2, 3, 5


def test_step_refusals(tpc):
    for name in ("q", "k", "v", "g", "beta", "o", "state", "src"):
        assert step(tpc, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "g", "o", "state"):
        assert step(tpc, **{name: A + 8}) == SHAPE, name
    assert step(tpc, d=96) == UNSUP and step(tpc, dv=64) == SHAPE and step(tpc, H=0) == SHAPE
    assert step(tpc, din=2) == UNSUP and step(tpc, dout=5) == UNSUP
    assert step(tpc, n_slots=-1) == SHAPE
    assert step(tpc, rws=rows(tpc, n=-1)) == SHAPE and step(tpc, rws=rows(tpc, seqs=-1)) == SHAPE
    assert step(tpc, rws=rows(tpc, n=5)) == SHAPE  # five rows of four sequences need row_start
    assert step(tpc, rws=rows(tpc, n=2**31 - 1, seqs=2**31 - 1), H=2**20) == SHAPE
    assert step(tpc, rws=rows(tpc, 0, 0), q=None, src=None, state=None) == 0  # nothing to do
    L = tpc.lib()
    assert L.tpc_kda_step(None, rows(tpc), C.byref(tpc.KdaStepIO()), None, None) == NULL
    assert L.tpc_kda_step(C.byref(tpc.KdaShape(1, 64, 64, 0, 0)), None, C.byref(tpc.KdaStepIO()), None, None) == NULL
    assert b"kda step" in L.tpc_last_error()


def test_append_refusals(tpc):
    L = tpc.lib()
    call = lambda c=None, r=None, x=A, ld=512, kr=A, ldk=64, dt=1: L.tpc_latent_append(
        c or cache(tpc), r or rows(tpc), x, ld, kr, ldk, dt, None, None)
    assert L.tpc_latent_append(None, rows(tpc), A, 512, A, 64, 1, None, None) == NULL
    assert L.tpc_latent_append(cache(tpc), None, A, 512, A, 64, 1, None, None) == NULL
    assert call(x=None) == NULL and call(kr=None) == NULL and call(r=rows(tpc, kv=None)) == NULL
    assert call(c=cache(tpc, data=None)) == NULL and call(c=cache(tpc, table=None)) == NULL
    assert call(c=cache(tpc, data=A + 2)) == SHAPE and call(x=A + 4) == SHAPE and call(kr=A + 4) == SHAPE
    assert call(ld=504) == SHAPE and call(ld=516) == SHAPE and call(ldk=60) == SHAPE and call(ld=514, dt=0) == SHAPE
    for page in (0, 1, 8, 17, 48, 65, 96, -64):
        assert call(c=cache(tpc, page=page)) == UNSUP, page
    assert call(c=cache(tpc, n_pages=0)) == SHAPE and call(c=cache(tpc, max_pages=0)) == SHAPE
    assert call(c=cache(tpc, n_pages=2**26)) == SHAPE and call(c=cache(tpc, max_pages=2**26)) == SHAPE
    assert call(c=cache(tpc, page=2**31 - 64, n_pages=1, max_pages=1)) == SHAPE  # a tile past the end must not wrap
    assert call(dt=2) == UNSUP and call(r=rows(tpc, n=3)) == SHAPE
    assert call(r=rows(tpc, 0, 0, kv=None), x=None, kr=None) == 0


def test_absorb_expand_refusals(tpc):
    L = tpc.lib()
    ab = lambda r=None, H=4, q=A, ld=768, w=A, qa=A: L.tpc_latent_absorb(r or rows(tpc), H, q, ld, w, qa, None, None)
    assert ab(q=None) == NULL and ab(w=None) == NULL and ab(qa=None) == NULL and ab(r=rows(tpc, kv=None)) == NULL
    assert ab(q=A + 2) == SHAPE and ab(w=A + 2) == SHAPE and ab(qa=A + 2) == SHAPE
    assert ab(ld=760) == SHAPE and ab(ld=772) == SHAPE
    assert ab(H=0) == UNSUP and ab(H=129, ld=129 * 192) == UNSUP
    assert ab(r=rows(tpc, n=2**25, seqs=2**25), H=64, ld=64 * 192) == SHAPE
    assert ab(r=rows(tpc, 0, 0, kv=None), q=None) == 0
    ex = lambda n=4, H=4, o=A, w=A, out=A: L.tpc_latent_expand(n, H, o, w, out, None, None)
    assert ex(o=None) == NULL and ex(w=None) == NULL and ex(out=None) == NULL
    assert ex(o=A + 2) == SHAPE and ex(w=A + 2) == SHAPE and ex(out=A + 2) == SHAPE
    assert ex(n=-1) == SHAPE and ex(H=0) == UNSUP and ex(H=129) == UNSUP and ex(n=2**25, H=64) == SHAPE
    assert ex(n=0, o=None) == 0


def test_attention_refusals(tpc):
    L = tpc.lib()
    nb = L.tpc_latent_attn_scratch_bytes(4)
    assert nb > 0 and L.tpc_latent_attn_scratch_bytes(0) == 0 and L.tpc_latent_attn_scratch_bytes(129) == 0
    at = lambda c=None, r=None, H=4, qa=A, o=A, lse=A, s=A, n=nb: L.tpc_latent_attn(
        c or cache(tpc), r or rows(tpc), H, 0.1, qa, o, lse, s, n, None, None)
    for name in ("qa", "o", "lse", "s"):
        assert at(**{name: None}) == NULL, name
    assert at(qa=A + 8) == SHAPE and at(o=A + 8) == SHAPE
    assert at(n=nb - 1) == WS and at(s=A + 16) == WS
    assert at(H=0) == UNSUP and at(H=129) == UNSUP and at(c=cache(tpc, page=40)) == UNSUP
    assert at(r=rows(tpc, kv=None)) == NULL and at(r=rows(tpc, n=3)) == SHAPE
    assert at(r=rows(tpc, 0, 0, kv=None), qa=None) == 0


def test_empty_batches_need_no_block_table(tpc):
    """A table of no sequence has no memory (an empty tensor's address is NULL)."""
    L = tpc.lib()
    ap = lambda c, r: L.tpc_latent_append(c, r, None, 512, None, 64, 1, None, None)
    at = lambda c, r: L.tpc_latent_attn(c, r, 4, 0.1, None, None, None, None, 0, None, None)
    for call in (ap, at):
        for r in ((0, 0, None, None), (0, 0, A, None), (3, 0, A, None)):
            assert call(cache(tpc, table=None), rows(tpc, *r)) == 0
            assert call(cache(tpc, table=None, max_pages=0), rows(tpc, *r)) == 0
            assert call(cache(tpc, data=None), rows(tpc, *r)) == NULL
            assert call(cache(tpc, max_pages=-1), rows(tpc, *r)) == SHAPE
        assert call(cache(tpc, table=None), rows(tpc, 0, 3, A)) == 0
        assert call(cache(tpc, table=None), rows(tpc, 3, 3)) == NULL


def test_wrappers_refuse_cpu_tensors(tpc):
    import torch
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(tpc.TpcError):
        x = z(1, 2, 64)
        tpc.tpc_kda_step(z(2, 2, 64, 64, t=torch.float32), i(1), x, x, x, x, z(1, 2))
    with pytest.raises(tpc.TpcError):
        tpc.tpc_latent_append(z(2, 64, 576), i(1, 2), i(1), z(1, 512), z(1, 64))
    with pytest.raises(tpc.TpcError):
        tpc.tpc_latent_absorb(z(1, 2, 192), z(512, 512), i(1))
    with pytest.raises(tpc.TpcError):
        tpc.tpc_latent_attn(z(1, 2, 576), z(2, 64, 576), i(1, 2), i(1), 0.1)
    with pytest.raises(tpc.TpcError):
        tpc.tpc_latent_expand(z(1, 2, 512), z(512, 512))


def test_oracle_absorbed_equals_expanded():
    """The absorbed oracle (append, absorb, attention, expand) is the expanded causal attention."""
    rng = np.random.default_rng(3)
    T, H, page = 37, 3, 16
    q, c, kr = rng.normal(size=(T, H, 192)), rng.normal(size=(T, 512)), rng.normal(size=(T, 64))
    w = 0.05 * rng.normal(size=(2 * H * 128, 512))
    table = np.array([[4, 0, 2]])
    cch = np.full((5, page, 576), np.nan)
    kv, start = np.array([T]), np.array([0, T])
    cch = od.append(cch, table, kv, c, kr, start)
    qa, _ = od.absorb(q, w, kv, start)
    o, lse, _, _ = od.attention(qa, cch, table, kv, 0.07, start)
    out, _ = od.expand(o, w)
    assert np.abs(out - od.expanded_attention(q, c, kr, w, 0.07)).max() < 1e-12


def test_oracle_step_equals_tree_recurrence():
    """The step oracle over a whole trajectory is the tree oracle's recurrence."""
    import synth
    from oracle import kda as okda
    w = synth.workload("fig1")
    inputs = synth.kda_inputs(5, np.arange(w.tree.n_rows), 2, 32, 32, "f32")
    o_ref, fin_ref = okda.tree_forward(w.tree, inputs)
    st = w.tree.node_start()
    leaf = w.tree.leaves()[1]
    idx = np.concatenate([np.arange(st[v], st[v] + w.tree.length[v]) for v in w.tree.path(leaf)])
    q, k, v, g, b = (x[idx].astype(np.float64) for x in inputs)
    o, new, _, _ = od.kda_step(np.zeros((1, 2, 32, 32)), [0], [0], q, k, v, g, b, np.array([0, len(idx)]))
    assert np.abs(o - o_ref[idx]).max() < 1e-12 and np.abs(new[0] - fin_ref[1]).max() < 1e-12


def test_packed_structs_have_the_c_layout(tpc):
    """The wrappers pack the C structs as bytes: the same fields as the ctypes classes, at the same offsets."""
    def same(cls, packed, *values):
        want = cls(*values)
        assert packed == bytes(want), cls
    same(tpc.Rows, tpc._pack_rows(3, 2, A, 2 * A), 3, 2, A, 2 * A)
    same(tpc.LatentCache, tpc._pack_cache(A, 5, 64, 2 * A, 7), A, 5, 64, 2 * A, 7)
    same(tpc.KdaStepIO, tpc._pack_step(*range(1, 7), 9, 10, 0, 11), *range(1, 7), 9, 10, 0, 11)
    same(tpc.KdaShape, tpc._pack_shape(2, 128, 128, True, False), 2, 128, 128, 1, 0)
