"""Tree decoding, without a GPU: refusals of the C entry points and of the
binding, size helpers, and the reference's own rejection sampling against the
law it has to keep."""
import ctypes
import random

import pytest
import torch

from tests import tree_ref as R

A, ODD, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001), ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def G():
    from latent_kv_cache_flash_b200 import build, gqla
    build.build()
    return gqla


def _dims(lib, **kw):
    base = dict(n_h=32, G=8, d_nope=128, d_rope=64, d_v=128, r=512, s_q=16, scale=192 ** -0.5, dtype=lib.GQLA_BF16, k_layout=0)
    base.update(kw)
    return lib.GqlaDims(*base.values())


def _layout(G, B=4, L=8192):
    lens = torch.full((B,), L, dtype=torch.int32)
    return lens, G.make_layout(lens, L, 0, L)


@pytest.mark.parametrize("path", ["gqa", "absorb"])
def test_decode_refusals(G, path):
    _, lay = _layout(G)
    big = 1 << 34
    tree = G.GqlaTree(A, None)

    def call(d, t=tree, q=A, out=A, ws=A, wsn=big, layout=lay, pool=A):
        p = ctypes.byref
        t = None if t is None else p(t)
        if path == "gqa":
            return G.lib().gqla_decode_tree_gqa(p(d), p(layout), t, q, pool, pool, out, None, 0, ws, wsn, None, None)
        return G.lib().gqla_decode_tree_absorb(p(d), p(layout), t, q, pool, A, A, out, None, 0, ws, wsn, None, None)

    for s_q in (0, 65, -1):
        assert call(_dims(G, s_q=s_q)) == G.GQLA_ERR_INVALID_ARG
    d = _dims(G)
    assert call(d, t=None) == G.GQLA_ERR_INVALID_ARG
    assert call(d, t=G.GqlaTree(None, A)) == G.GQLA_ERR_INVALID_ARG
    assert call(d, q=NULL) == G.GQLA_ERR_INVALID_ARG
    assert call(d, pool=NULL) == G.GQLA_ERR_INVALID_ARG
    assert call(d, q=ctypes.c_void_p(0x10008)) == G.GQLA_ERR_ALIGNMENT
    assert call(d, out=ctypes.c_void_p(0x10004)) == G.GQLA_ERR_ALIGNMENT
    assert call(_dims(G, G=5)) == G.GQLA_ERR_INVALID_ARG
    assert call(_dims(G, r=700, d_nope=700)) == G.GQLA_ERR_UNSUPPORTED
    kind = G.GQLA_PATH_GQA if path == "gqa" else G.GQLA_PATH_ABSORB
    need = G.gqla_tree_workspace_bytes(d, lay, 0, kind)
    if need:
        assert call(d, wsn=need - 1) == G.GQLA_ERR_WORKSPACE
        assert call(d, ws=NULL) == G.GQLA_ERR_WORKSPACE
        assert call(d, ws=ctypes.c_void_p(0x10010)) == G.GQLA_ERR_WORKSPACE


def test_sizes_follow_the_slots(G):
    _, lay = _layout(G, B=2, L=4000)
    for path in (G.GQLA_PATH_GQA, G.GQLA_PATH_ABSORB):
        for s_q in (1, 5, 64):
            d = _dims(G, s_q=s_q)
            S = G.gqla_tree_num_splits(d, lay, 0, path)
            assert S >= 1
            ws = G.gqla_tree_workspace_bytes(d, lay, 0, path)
            if S > 1:
                width = 128 if path == G.GQLA_PATH_GQA else 512
                assert ws >= S * 2 * s_q * 32 * (width + 1) * 4
        assert G.gqla_tree_workspace_bytes(_dims(G, s_q=65), lay, 0, path) == 0
        assert G.gqla_tree_num_splits(_dims(G, s_q=65), lay, 0, path) == 0
    # the causal calls keep their range
    assert G.gqla_num_splits(_dims(G, s_q=5), lay, 0, G.GQLA_PATH_GQA) == 0


def test_masks_append_refusals(G):
    L = G.lib()
    assert L.gqla_tree_masks(0, 4, A, None, A, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_tree_masks(2, 0, A, None, A, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_tree_masks(2, 65, A, None, A, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_tree_masks(2, 4, NULL, None, A, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_tree_masks(2, 4, A, None, NULL, None, None) == G.GQLA_ERR_INVALID_ARG
    _, lay = _layout(G)
    d, p = _dims(G), ctypes.byref
    assert L.gqla_append_tree(p(d), p(lay), None, NULL, A, A, A, A, A, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_append_tree(p(d), p(lay), None, A, NULL, A, A, NULL, NULL, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_append_tree(p(d), p(lay), None, A, A, A, A, A, NULL, None, None) == G.GQLA_ERR_INVALID_ARG
    assert L.gqla_append_tree(p(d), p(lay), None, ODD, A, A, A, A, A, None, None) == G.GQLA_ERR_ALIGNMENT
    d = _dims(G, s_q=65)
    assert L.gqla_append_tree(p(d), p(lay), None, A, A, A, A, A, A, None, None) == G.GQLA_ERR_INVALID_ARG


def test_verify_refusals(G):
    def call(batch=2, n=4, vocab=100, parents=A, tokens=A, target=A, tp=100, draft=A, dp=100, dt=0, ua=A, us=A, acc=A,
             na=A, nt=A):
        return G.lib().gqla_verify_tree(batch, n, vocab, parents, None, tokens, target, tp, draft, dp, dt, ua, us, acc,
                                        na, nt, None, None)
    bad = G.GQLA_ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(n=0), dict(n=65), dict(vocab=0), dict(tp=99), dict(dp=99), dict(dt=2)):
        assert call(**kw) == bad, kw
    for name in ("parents", "tokens", "target", "ua", "us", "acc", "na", "nt"):
        assert call(**{name: NULL}) == bad, name
    assert call(target=ctypes.c_void_p(0x10002)) == G.GQLA_ERR_ALIGNMENT
    assert call(draft=ctypes.c_void_p(0x10002)) == G.GQLA_ERR_ALIGNMENT
    assert call(draft=ODD, dt=1) == G.GQLA_ERR_ALIGNMENT


def test_commit_refusals(G):
    _, lay = _layout(G)
    seq = ctypes.c_void_p(lay.seq_lens)

    def call(n=4, acc=A, na=A, pools=((0x10000, 64),), out=A, layout=lay, count=None):
        arr = (G.GqlaPool * max(1, len(pools)))(*[G.GqlaPool(*x) for x in pools])
        return G.lib().gqla_commit_tree(ctypes.byref(layout), n, None, acc, na, arr, len(pools) if count is None else count,
                                        out, None, None)
    bad = G.GQLA_ERR_INVALID_ARG
    for kw in (dict(n=0), dict(n=65), dict(acc=NULL), dict(na=NULL), dict(count=0), dict(pools=((None, 64),)),
               dict(pools=((0x10000, 0),)), dict(out=seq)):
        assert call(**kw) == bad, kw
    assert call(pools=((0x10001, 64),)) == G.GQLA_ERR_ALIGNMENT
    assert call(pools=((0x10000, 64), (0x20000, 33))) == G.GQLA_ERR_ALIGNMENT
    assert call(layout=G.make_layout(torch.ones(2, dtype=torch.int32), 0, 0, 8)) == bad


def test_binding_checks_shapes_and_types(G):
    i32 = dict(dtype=torch.int32)
    good = dict(parents=torch.zeros(2, 3, **i32), tokens=torch.zeros(2, 3, **i32), target=torch.zeros(2, 3, 7), draft=None,
                u_accept=torch.zeros(2, 3), u_sample=torch.zeros(2), accepted=torch.zeros(2, 3, **i32),
                n_accepted=torch.zeros(2, **i32), next_token=torch.zeros(2, **i32))
    for name, t in (("parents", torch.zeros(2, 3)), ("tokens", torch.zeros(2, 4, **i32)),
                    ("target", torch.zeros(2, 3, 7, dtype=torch.float16)), ("target", torch.zeros(2, 7, 3).transpose(1, 2)),
                    ("draft", torch.zeros(2, 3, 7, dtype=torch.bfloat16)), ("draft", torch.zeros(2, 3, 8)),
                    ("target", torch.zeros(2, 4, 7)[:, :3]),
                    ("u_accept", torch.zeros(3, 2).t()), ("u_sample", torch.zeros(2, dtype=torch.float64)),
                    ("accepted", torch.zeros(3, 2, **i32).t()), ("n_accepted", torch.zeros(3, **i32)),
                    ("next_token", torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            G.gqla_verify_tree(**{**good, name: t})
    with pytest.raises(ValueError):
        G.make_tree(torch.zeros(2, 3, **i32))
    with pytest.raises(ValueError):
        G.make_tree(torch.zeros(2, 3, dtype=torch.int64), torch.zeros(3, **i32))
    with pytest.raises(ValueError):
        G.gqla_tree_masks(torch.zeros(2, 3, **i32), torch.zeros(2, 4, dtype=torch.int64))
    lay = G.make_layout(torch.ones(2, **i32), 8, 0, 8)
    acc, n = torch.zeros(2, 3, **i32), torch.zeros(2, **i32)
    for pools in ([], [torch.zeros(2, 9, 4)], [torch.zeros(2, 4, 8).transpose(1, 2)]):
        with pytest.raises(ValueError):
            G.gqla_commit_tree(lay, acc, n, pools)
    with pytest.raises(ValueError):
        G.gqla_commit_tree(lay, torch.zeros(3, 3, **i32), n, [torch.zeros(2, 8, 4)])


@pytest.mark.parametrize("shape", ["chain", "star"])
def test_reference_sampling_keeps_the_targets_law(shape):
    """The first token after the root (an accepted draft or the one drawn) is
    distributed as the target: 40000 seeded trials, five standard deviations."""
    rng = random.Random(7)
    target = [[0.5, 0.3, 0.15, 0.05], [0.1, 0.2, 0.3, 0.4], [0.25] * 4, [0.7, 0.1, 0.1, 0.1]]
    draft = [[0.2, 0.2, 0.5, 0.1], [0.4, 0.3, 0.2, 0.1], [0.25] * 4, [0.1, 0.2, 0.3, 0.4]]
    parents = [-1, 0, 1, 2] if shape == "chain" else [-1, 0, 0, 0]
    trials, count = 40000, [0] * 4
    for _ in range(trials):
        tokens = [0] + [rng.choices(range(4), draft[parents[j]])[0] for j in range(1, 4)]
        path, nxt = R.verify(parents, 4, tokens, target, draft, [rng.random() for _ in range(4)], rng.random())
        count[tokens[path[1]] if len(path) > 1 else nxt] += 1
    for v, p in enumerate(target[0]):
        assert abs(count[v] - trials * p) < 5 * (trials * p * (1 - p)) ** 0.5


def _attention_args(G, path, dtype=torch.bfloat16, page=0, shared=0):
    B, T, h, g, n, r, v, R, L = 2, 3, 4, 2, 16, 8, 24, 32, 64
    d = G.GqlaDims(h, g, n, r, v, R, T, 0.1, G.GQLA_BF16 if dtype is torch.bfloat16 else G.GQLA_F32, shared)
    lens = torch.full((B,), 10, dtype=torch.int32)
    lead = (5, page) if page else (B, L)
    table = torch.zeros((B, 2), dtype=torch.int32) if page else None
    lay = G.make_layout(lens, L, page, 0 if page else L, table, 5 if page else 0)
    a = dict(dims=d, layout=lay, tree=G.make_tree(torch.zeros((B, T), dtype=torch.int64)),
             q=torch.zeros((B, T, h, n + r), dtype=dtype), out=torch.zeros((B, T, h, v), dtype=dtype),
             lse=torch.zeros((B, T, h)))
    weights = dict(W_uk=torch.zeros((g, R, n), dtype=dtype), W_uv=torch.zeros((g, R, v), dtype=dtype))
    pools = dict(k_pool=torch.zeros(lead + ((g * n + r,) if shared else (g, n + r)), dtype=dtype),
                 v_pool=torch.zeros(lead + (g, v), dtype=dtype))
    latent = dict(latent=torch.zeros(lead + (R + r,), dtype=dtype))
    if path == "append":
        a = dict(dims=d, layout=lay, new_rows=torch.zeros((B, T, R + r), dtype=dtype), sizes=None)
        return {**a, **latent, **weights, **pools}
    return {**a, **(pools if path == "gqa" else {**latent, **weights})}


@pytest.mark.parametrize("path", ["gqa", "absorb", "append"])
@pytest.mark.parametrize("page,shared,dtype", [(0, 0, torch.bfloat16), (16, 1, torch.float32)])
def test_binding_checks_the_attentions_tensors(G, path, page, shared, dtype):
    """Masks of another tree or batch, and any tensor of another type, size or
    order, are refused before the library is called."""
    call = {"gqa": G.gqla_decode_tree_gqa, "absorb": G.gqla_decode_tree_absorb, "append": G.gqla_append_tree}[path]
    good = _attention_args(G, path, dtype, page, shared)
    wrong = []
    for name, t in good.items():
        if isinstance(t, torch.Tensor):
            wrong += [(name, t.to(torch.float16)), (name, t[:-1]), (name, t.transpose(0, 1))]
            if "pool" not in name and name != "latent":
                wrong.append((name, torch.cat([t, t])))
    i64 = dict(dtype=torch.int64)
    if path == "append":
        wrong += [("sizes", torch.zeros(3, dtype=torch.int32)), ("sizes", torch.zeros(2, **i64))]
    else:
        wrong += [("tree", G.make_tree(torch.zeros(shape, **i64))) for shape in ((2, 2), (2, 4), (1, 3), (3, 2))]
        wrong += [("workspace", torch.zeros((64, 64), dtype=torch.uint8).t())]
    wrong += [("dev_status", torch.zeros(1, **i64)), ("dev_status", torch.zeros(0, dtype=torch.int32))]
    for name, t in wrong:
        with pytest.raises(ValueError):
            call(**{**good, name: t})
    # what is right gets past the checks: the library itself refuses these dims
    good["dims"].scale = float("nan")
    with pytest.raises(G.GqlaError):
        call(**good)


def test_a_requested_split_count_has_a_limit(G):
    """256 splits at most, however many tiles there are and more are asked for,
    and no more workspace for asking; the library's own choice is 64 at most."""
    for L in (64000, 10 ** 6, 2 ** 31 - 1):
        _, lay = _layout(G, B=1, L=L)
        d = _dims(G, n_h=2, G=2, d_nope=16, d_rope=8, d_v=16, r=32, s_q=2, dtype=G.GQLA_F32)
        for path in (G.GQLA_PATH_GQA, G.GQLA_PATH_ABSORB):
            counts = [G.gqla_tree_num_splits(d, lay, n, path) for n in (1, 255, 256, 257, 900, 2000, 2 ** 31 - 1)]
            assert counts[0] == 1 and max(counts) <= 256 and counts == sorted(counts)
            assert len({G.gqla_tree_workspace_bytes(d, lay, n, path) for n in (256, 900, 2000, 2 ** 31 - 1)}) == 1
            assert 1 <= G.gqla_tree_num_splits(d, lay, 0, path) <= 64
    # fewer tiles than asked for
    _, lay = _layout(G, B=1, L=130)
    assert G.gqla_tree_num_splits(d, lay, 2000, G.GQLA_PATH_GQA) == 3


def test_arrays_off_their_elements_size_are_refused(G):
    """A read of them would be a misaligned access on the device."""
    L, p = G.lib(), ctypes.byref
    at = lambda off: ctypes.c_void_p(0x10000 + off)     # noqa: E731
    off2, off4 = at(2), at(4)
    no = G.GQLA_ERR_ALIGNMENT
    lens, lay = _layout(G)
    d = _dims(G)
    far = _layout(G)[1]
    far.seq_lens = 0x10002
    for call in (lambda t=p(G.GqlaTree(at(0), None)), lse=None, st=None, lay=lay:
                 L.gqla_decode_tree_gqa(p(d), p(lay), t, A, A, A, A, lse, 0, A, 1 << 34, st, None),
                 lambda t=p(G.GqlaTree(at(0), None)), lse=None, st=None, lay=lay:
                 L.gqla_decode_tree_absorb(p(d), p(lay), t, A, A, A, A, A, lse, 0, A, 1 << 34, st, None)):
        for kw in (dict(t=p(G.GqlaTree(off4, None))), dict(t=p(G.GqlaTree(A, off2))), dict(lse=off2), dict(st=off2), dict(lay=far)):
            assert call(**kw) == no, kw
    assert L.gqla_append_tree(p(d), p(lay), off2, A, A, A, A, A, A, None, None) == no
    assert L.gqla_append_tree(p(d), p(lay), None, A, A, A, A, A, A, off2, None) == no
    assert L.gqla_append_tree(p(d), p(far), None, A, A, A, A, A, A, None, None) == no
    for args in ((off2, None, A, None), (A, off2, A, None), (A, None, off4, None), (A, None, A, off2)):
        assert L.gqla_tree_masks(2, 4, *args, None) == no
    good = [A, A, A, A, 100, A, 100, 0, A, A, A, A, A, A]
    for i in (0, 1, 2, 8, 9, 10, 11, 12, 13):
        args = list(good)
        args[i] = off2
        assert L.gqla_verify_tree(2, 4, 100, *args, None) == no, i
    pool = (G.GqlaPool * 1)(G.GqlaPool(0x10000, 64))
    for sizes, acc, n, out, st, l in ((off2, A, A, A, None, lay), (None, off2, A, A, None, lay), (None, A, off2, A, None, lay),
                                      (None, A, A, off2, None, lay), (None, A, A, A, off2, lay), (None, A, A, A, None, far)):
        assert L.gqla_commit_tree(p(l), 4, sizes, acc, n, pool, 1, out, st, None) == no
