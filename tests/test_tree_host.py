"""Host-side checks of the tree-drafting entry points: every bad argument is
refused before anything is enqueued (no GPU here: a call that reached a launch
would return SV_ERR_HIP), workspace queries, and the binding's own checks."""
import ctypes
import math
import os

import numpy as np
import pytest

import speculative_decoding_verification_amd as sv
from speculative_decoding_verification_amd import tree

ST = sv.STATUS_CODE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.library_path()):
        pytest.fail("libspecverify.so is not built; run __graft_entry__.build()")
    return sv.load_library()


def attn_desc(**over):
    f = dict(B=2, k=5, q_heads=8, kv_heads=2, head_dim=128, n_pages=10, page_size=16, max_pages=4, dtype=sv.SV_BF16,
             scale=0.1, q_stride_b=6 * 8 * 128, q_stride_r=8 * 128, q_stride_h=128)
    f.update(over)
    return tree.TreeAttentionDesc(**f)


def attn_call(lib, desc, ptr=None, ws_bytes=None, **over):
    names = ["q", "k_cache", "v_cache", "page_table", "seq_len", "parents", "out", "lse", "workspace"]
    a = {n: 1 << 20 for n in names}
    a.update(over)
    n = lib.sv_tree_attention_workspace_bytes(ctypes.byref(desc)) if ws_bytes is None else ws_bytes
    return lib.sv_tree_attention(ctypes.byref(desc), *[a[x] for x in names], n, None)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, "BAD_SHAPE"), ("B", 65536, "BAD_SHAPE"), ("k", -1, "BAD_SHAPE"), ("k", 65, "BAD_SHAPE"),
    ("q_heads", 0, "BAD_SHAPE"), ("q_heads", 7, "BAD_SHAPE"), ("q_heads", 1026, "BAD_SHAPE"), ("kv_heads", 0, "BAD_SHAPE"),
    ("kv_heads", 3, "BAD_SHAPE"), ("head_dim", 80, "BAD_SHAPE"), ("head_dim", 0, "BAD_SHAPE"), ("n_pages", 0, "BAD_SHAPE"),
    ("page_size", 0, "BAD_SHAPE"), ("page_size", 24, "BAD_SHAPE"), ("page_size", 2048, "BAD_SHAPE"),
    ("max_pages", 0, "BAD_SHAPE"), ("max_pages", (1 << 26) + 1, "BAD_SHAPE"), ("n_pages", 1 << 27, "BAD_SHAPE"),
    ("dtype", sv.SV_F32, "BAD_DTYPE"), ("dtype", 3, "BAD_DTYPE"), ("scale", 0.0, "BAD_SCALE"), ("scale", -1.0, "BAD_SCALE"),
    ("scale", math.inf, "BAD_SCALE"), ("scale", math.nan, "BAD_SCALE"), ("q_stride_h", 4, "MISALIGNED"),
    ("q_stride_r", -8, "MISALIGNED"), ("q_stride_b", 7, "MISALIGNED")])
def test_attention_rejects_bad_desc(lib, field, value, status):
    d = attn_desc(**{field: value})
    assert lib.sv_tree_attention_workspace_bytes(ctypes.byref(d)) == 0
    assert attn_call(lib, d, ws_bytes=1 << 30) == ST["SV_ERR_" + status]


def test_attention_rejects_bad_arguments(lib):
    d = attn_desc()
    for name in ("q", "k_cache", "v_cache", "page_table", "seq_len", "parents", "out", "workspace"):
        assert attn_call(lib, d, **{name: None}) == ST["SV_ERR_NULL_ARG"], name
    for name in ("q", "k_cache", "v_cache", "out", "workspace"):
        assert attn_call(lib, d, **{name: (1 << 20) + 8}) == ST["SV_ERR_MISALIGNED"], name
    n = lib.sv_tree_attention_workspace_bytes(ctypes.byref(d))
    assert n >= 256
    assert attn_call(lib, d, ws_bytes=n - 1) == ST["SV_ERR_WORKSPACE_TOO_SMALL"]
    assert lib.sv_tree_attention(None, *[1 << 20] * 9, n, None) == ST["SV_ERR_NULL_ARG"]
    assert lib.sv_tree_attention_workspace_bytes(None) == 0
    empty = attn_desc(B=0)
    assert attn_call(lib, empty, **{x: None for x in ("q", "k_cache", "out", "workspace")}) == ST["SV_OK"]


def test_attention_rejects_output_on_its_queries(lib):
    assert attn_call(lib, attn_desc(), out=1 << 20, q=1 << 20) == ST["SV_ERR_ALIASED"]


def tree_desc(**over):
    f = dict(B=2, k=5, V=100, draft_rows=4, dtype=sv.SV_BF16, draft_kind=sv.SV_DRAFT_LOGITS, temperature=1.0)
    f.update(over)
    return tree.VerifyTreeDesc(**f)


def tree_call(lib, desc, ws_bytes=None, **over):
    names = ["target", "draft", "tokens", "parents", "uniforms", "accepted_len", "out_tokens", "path", "workspace"]
    a = {n: 1 << 20 for n in names}
    a.update(over)
    n = lib.sv_verify_tree_workspace_bytes(ctypes.byref(desc)) if ws_bytes is None else ws_bytes
    return lib.sv_verify_tree(ctypes.byref(desc), *[a[x] for x in names], n, None)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, "BAD_SHAPE"), ("k", 0, "BAD_SHAPE"), ("k", 65, "BAD_SHAPE"), ("V", 0, "BAD_SHAPE"),
    ("V", (1 << 24) + 1, "BAD_SHAPE"), ("draft_rows", 0, "BAD_SHAPE"), ("draft_rows", 7, "BAD_SHAPE"),
    ("dtype", sv.SV_F16, "BAD_DTYPE"), ("draft_kind", 2, "BAD_DRAFT_KIND"), ("temperature", -1.0, "BAD_TEMPERATURE"),
    ("temperature", 1e-5, "BAD_TEMPERATURE"), ("temperature", math.nan, "BAD_TEMPERATURE"),
    ("temperature", math.inf, "BAD_TEMPERATURE")])
def test_walk_rejects_bad_desc(lib, field, value, status):
    d = tree_desc(**{field: value})
    assert lib.sv_verify_tree_workspace_bytes(ctypes.byref(d)) == 0
    assert tree_call(lib, d, ws_bytes=1 << 30) == ST["SV_ERR_" + status]


def test_walk_rejects_bad_arguments(lib):
    d = tree_desc()
    for name in ("target", "draft", "tokens", "parents", "uniforms", "accepted_len", "out_tokens", "path", "workspace"):
        assert tree_call(lib, d, **{name: None}) == ST["SV_ERR_NULL_ARG"], name
    assert tree_call(lib, d, workspace=(1 << 20) + 32) == ST["SV_ERR_MISALIGNED"]
    assert tree_call(lib, d, target=(1 << 20) + 1) == ST["SV_ERR_MISALIGNED"]
    n = lib.sv_verify_tree_workspace_bytes(ctypes.byref(d))
    assert tree_call(lib, d, ws_bytes=n - 1) == ST["SV_ERR_WORKSPACE_TOO_SMALL"]
    assert tree_call(lib, tree_desc(B=0), target=None, workspace=None) == ST["SV_OK"]
    # greedy and one-hot calls read no draft rows
    assert lib.sv_verify_tree_workspace_bytes(ctypes.byref(tree_desc(draft_rows=0, temperature=0.0))) >= 256
    assert lib.sv_verify_tree_workspace_bytes(ctypes.byref(tree_desc(draft_rows=-3, draft_kind=sv.SV_DRAFT_ONEHOT))) >= 256


def cache_desc(**over):
    f = dict(n_seqs=3, n_pages=10, page_size=16, max_pages=4, n_layers=2, kv_heads=2, head_dim=64, dtype=sv.SV_F16)
    f.update(over)
    return tree.CacheDesc(**f)


ROWS = dict(t=4, k_stride_b=512, k_stride_t=128, k_stride_h=64, v_stride_b=512, v_stride_t=128, v_stride_h=64)
P = 1 << 20


def cache_calls(lib, d):
    """One call of each entry point, by name: (function, argument names, arguments)."""
    r = ctypes.byref(d)
    rows = tree.CacheRows(**ROWS)
    return {
        "append": (lib.sv_cache_append, ["k_new", "v_new", "count", "page_table", "seq_len", "k_cache", "v_cache"],
                   [r, ctypes.byref(rows)], [P, P, P, P, P, P, 2 * P], [None]),
        "commit": (lib.sv_cache_commit, ["path", "accepted_len", "page_table", "seq_len", "new_len", "k_cache", "v_cache"],
                   [r, 5], [P, P, P, P, 2 * P, P, 2 * P], [None]),
        "fork": (lib.sv_cache_fork, ["src", "dst", "page_table", "page_count", "page_refs", "seq_len", "k_cache", "v_cache",
                                     "status", "workspace"], [r, 3], [P, P, P, P, P, P, P, 2 * P, P, P], [1 << 20, None]),
        "resize": (lib.sv_cache_resize, ["want_len", "page_table", "page_count", "page_refs", "status"], [r],
                   [P, P, P, P, P], [None])}


@pytest.mark.parametrize("field,value,status", [
    ("n_seqs", -1, "BAD_SHAPE"), ("n_seqs", 4097, "BAD_SHAPE"), ("n_pages", 0, "BAD_SHAPE"), ("page_size", 12, "BAD_SHAPE"),
    ("max_pages", 0, "BAD_SHAPE"), ("max_pages", 1 << 27, "BAD_SHAPE"), ("n_layers", 0, "BAD_SHAPE"), ("kv_heads", 0, "BAD_SHAPE"),
    ("kv_heads", 1025, "BAD_SHAPE"), ("head_dim", 60, "BAD_SHAPE"), ("head_dim", 1032, "BAD_SHAPE"), ("dtype", sv.SV_F32, "BAD_DTYPE")])
def test_cache_rejects_bad_desc(lib, field, value, status):
    d = cache_desc(**{field: value})
    for name, (f, _, head, args, end) in cache_calls(lib, d).items():
        assert f(*head, *args, *end) == ST["SV_ERR_" + status], name
    assert lib.sv_cache_fork_workspace_bytes(ctypes.byref(d), 3) == 0


def test_cache_rejects_bad_arguments(lib):
    d = cache_desc()
    optional = {"count", "status"}
    for name, (f, names, head, args, end) in cache_calls(lib, d).items():
        for i, a in enumerate(names):
            if a not in optional:
                assert f(*head, *(args[:i] + [None] + args[i + 1:]), *end) == ST["SV_ERR_NULL_ARG"], (name, a)
            if a in ("k_new", "v_new", "k_cache", "v_cache"):
                assert f(*head, *(args[:i] + [P + 8] + args[i + 1:]), *end) == ST["SV_ERR_MISALIGNED"], (name, a)
        if "k_cache" in names:
            i = names.index("k_cache")
            same = args[:i] + [P, P] + args[i + 2:]
            assert f(*head, *same, *end) == ST["SV_ERR_ALIASED"], name
        assert f(None, *head[1:], *args, *end) == ST["SV_ERR_NULL_ARG"], name
    f, _, head, args, end = cache_calls(lib, d)["commit"]
    assert f(*head, *(args[:4] + [args[3]] + args[5:]), *end) == ST["SV_ERR_ALIASED"]
    for k in (0, 65):
        assert f(head[0], k, *args, *end) == ST["SV_ERR_BAD_SHAPE"]
    f, _, head, args, end = cache_calls(lib, d)["fork"]
    for n in (-1, 4097):
        assert f(head[0], n, *args, *end) == ST["SV_ERR_BAD_SHAPE"]
    need = lib.sv_cache_fork_workspace_bytes(ctypes.byref(d), 3)
    assert f(*head, *args, need - 1, None) == ST["SV_ERR_WORKSPACE_TOO_SMALL"]
    assert f(head[0], 0, *args, *end) == ST["SV_OK"]
    f, _, head, args, end = cache_calls(lib, d)["append"]
    for field in ROWS:
        rows = tree.CacheRows(**{**ROWS, field: -1 if field == "t" else 4})
        assert f(head[0], ctypes.byref(rows), *args, *end) == ST["SV_ERR_BAD_SHAPE" if field == "t" else "SV_ERR_MISALIGNED"]
    assert f(head[0], None, *args, *end) == ST["SV_ERR_NULL_ARG"]
    none = cache_desc(n_seqs=0)
    for name, (f, _, head, args, end) in cache_calls(lib, none).items():
        if name != "fork":
            assert f(*head, *args, *end) == ST["SV_OK"], name


def test_attention_workspace_depends_on_rows_not_on_batch(lib):
    n = lambda **o: lib.sv_tree_attention_workspace_bytes(ctypes.byref(attn_desc(**o)))  # noqa: E731
    assert n(B=1) == n(B=500) and n(k=0) <= n(k=5) <= n(k=64)


def test_binding_checks(lib):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    q = torch.zeros((3, 5, 4, 64), dtype=torch.bfloat16)
    good = dict(q=q, k_cache=kc, v_cache=kc.clone(), page_table=i32(3, 2), seq_len=i32(3), parents=i32(3, 4))
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=kc[0]), dict(v_cache=kc[:3]), dict(page_table=i32(2, 2)),
                dict(seq_len=i32(3).long()), dict(parents=i32(3, 5)), dict(parents=None), dict(q=q.transpose(2, 3)),
                dict(k_cache=kc[:, :, ::2]), dict(q=torch.zeros((3, 5, 4, 128), dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            tree.TreeAttention(**{**good, **bad})
    with pytest.raises(sv.SVError):
        tree.TreeAttention(**good, scale=-1.0)
    t, d = torch.zeros((3, 5, 10)), torch.zeros((3, 2, 10))
    good = dict(target=t, draft=d, draft_tokens=i32(3, 4), parents=i32(3, 4), uniforms=torch.zeros((3, 5)), temperature=1.0)
    for bad in (dict(target=t.double()), dict(draft=None), dict(draft=torch.zeros((3, 2, 9))), dict(draft=d.bfloat16()),
                dict(uniforms=None), dict(uniforms=torch.zeros((3, 4))), dict(parents=i32(3, 3)), dict(target=t[0])):
        with pytest.raises((ValueError, TypeError)):
            tree.TreeVerifier(**{**good, **bad})
    with pytest.raises(sv.SVError):
        tree.TreeVerifier(**{**good, "draft": torch.zeros((3, 6, 10))})
    k5 = torch.zeros((2, 4, 2, 16, 64), dtype=torch.float16)
    v5, n = k5.clone(), i32(3)
    for call in (lambda: tree.cache_append(q[:, :, :2], q[:, :, :2], kc, kc.clone(), i32(2, 2), i32(3)),
                 lambda: tree.cache_append(q[:, :, :2], q[:, :, :2, :32], kc, kc.clone(), i32(3, 2), i32(3)),
                 lambda: tree.cache_commit(i32(3, 4), i32(2), k5, v5, i32(3, 2), i32(3)),
                 lambda: tree.cache_fork(i32(2), i32(3), k5, v5, i32(3, 2), i32(3), i32(4), i32(3)),
                 lambda: tree.cache_resize(i32(2), i32(3, 2), i32(3), i32(4), page_size=16),
                 # everything fits, but these are host tensors
                 lambda: tree.tree_attention(**{**dict(q=q, k_cache=kc, v_cache=kc.clone(), page_table=i32(3, 2)),
                                                "seq_len": n, "parents": i32(3, 4)}),
                 lambda: tree.verify_tree(t, d, i32(3, 4), i32(3, 4), torch.zeros((3, 5)), 1.0),
                 lambda: tree.cache_append(q[:, :, :2], q[:, :, :2], kc, kc.clone(), i32(3, 2), n, stream=0),
                 lambda: tree.cache_commit(i32(3, 4), n, k5, v5, i32(3, 2), i32(3), stream=0),
                 lambda: tree.cache_resize(n, i32(3, 2), i32(3), i32(4), page_size=16, stream=0)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_reference_walk_is_lossless_by_enumeration():
    """The reference's rule against its purpose: over a fine grid of uniforms and all draws of two siblings from q, the
    first token's frequencies are p's."""
    import tree_reference as ref

    V, G = 3, 24
    p, q = np.array([0.2, 0.5, 0.3]), np.array([0.6, 0.1, 0.3])
    t, d = np.log(np.stack([p] * 3)), np.log(q)[None]
    grid = (np.arange(G) + 0.5) / G
    got = np.zeros(V)
    for x in range(V):
        for y in range(V):
            for u0 in grid:
                for u1 in grid:
                    for u2 in grid:
                        _, out, _, _ = ref.walk(t, d, [x, y], [-1, -1], [u0, u1, u2], 1.0, False)
                        got[out[0]] += q[x] * q[y] / G ** 3
    # each of the three uniforms is resolved to 1 / G
    assert np.abs(got - p).max() < 3.0 / G / 2
