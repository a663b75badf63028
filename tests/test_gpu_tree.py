"""Trees of drafted tokens and the paged cache on the GPU, against plain 64-bit
references (tree_reference.py): attention over odd sizes, masks, strides and
types, the walk in every mode, the cache's bookkeeping, and a whole decode
step, eager and as a replayed graph."""
import numpy as np
import pytest

import tree_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import speculative_decoding_verification_amd as sv  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a step of the type, relative
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    sv.load_library()
    return torch.device("cuda:0")


def trees(rs, B, k, absent=0.0):
    p = np.full((B, k), -1, np.int32)
    for b in range(B):
        for i in range(k):
            p[b, i] = rs.randint(max(-1, i - 6), i) if rs.rand() >= absent else -2
    return p


def paged(rs, tokens, page, spare=2, width=None):
    need = [-(-int(t) // page) if t > 0 else 0 for t in tokens]
    P = sum(need) + spare
    order = list(rs.permutation(P))
    table = np.full((len(need), width or max(1, max(need))), -1, np.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    return table, P


class Case:
    """Inputs of one attention call; dead slots hold NaN."""

    def __init__(self, dev, dtype="bf16", k=5, hq=8, hkv=2, D=128, page=16, lens=(37, 0, 130), seed=0, absent=0.0,
                 scale=None, amp=1.0, fill=float("nan")):
        rs = np.random.RandomState(seed)
        self.k, self.dtype, self.scale = k, dtype, scale or D ** -0.5
        B, t = len(lens), DT[dtype]
        self.table, P = paged(rs, [n + k + 1 for n in lens], page)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: (torch.randn(s, generator=g) * amp).to(t)  # noqa: E731
        self.q = rnd(B, k + 1, hq, D)
        self.kc, self.vc = rnd(P, hkv, page, D), rnd(P, hkv, page, D)
        self.parents = trees(rs, B, k, absent)
        live = np.zeros((P, page), bool)
        for b, n in enumerate(lens):
            if n < 0:
                continue
            see = ref.sees(self.parents[b], k)
            for pos in list(range(n)) + [n + j for j in range(k + 1) if see[j, j]]:
                live[self.table[b, pos // page], pos % page] = True
        dead = torch.from_numpy(~live)[:, None, :, None]
        self.kc.masked_fill_(dead, fill)
        self.vc.masked_fill_(dead, fill)
        self.lens = np.array(lens, np.int32)
        self.dev = dev

    def on(self, x):
        return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(self.dev)

    def args(self):
        return (self.on(self.q), self.on(self.kc), self.on(self.vc), self.on(self.table), self.on(self.lens),
                self.on(self.parents) if self.k else None)

    def check(self, out, lse):
        clean = lambda x: np.nan_to_num(x.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
        want, wlse, absv, dot = ref.attention(clean(self.q), clean(self.kc), clean(self.vc), self.table, self.lens,
                                              self.parents, self.scale)
        self.compare(out, lse, want, wlse, absv, dot)

    def compare(self, out, lse, want, wlse, absv, dot):
        """Bound: the output's rounding h |o|, the weights' roundings h sum p|v|, and the scores' 32-bit errors.  A
        score is a sum of D products whose partial sums are at most `dot`: off by at most D 2^-24 dot; its scaling,
        the exponent's argument and 2^x add 2^-22 (2 + |s|), |s| <= dot.  A relative error e of every weight moves
        the quotient by at most 2 e sum p|v|, and the sums of n weights and products add n 2^-24 each, n the keys."""
        u, h = 2.0 ** -24, HALF[self.dtype]
        D = self.q.shape[3]
        n = int(self.lens.max()) + self.k + 1
        e = (D + 2) * u * dot + 4 * u * (2 + dot)
        tol = h * (np.abs(want) + absv) * 1.01 + (2 * e + 2 * n * u)[..., None] * absv + 2.0 ** -24
        got = out.double().cpu().numpy()
        off = np.abs(got - want)
        assert np.isfinite(got).all()
        worst = (off / tol).max() if off.size else 0.0
        assert worst <= 1.0, "out: %.3g of the bound" % worst
        gl = lse.double().cpu().numpy()
        fin = np.isfinite(wlse)
        assert np.array_equal(np.isneginf(gl), ~fin)
        ltol = e + n * u + 2.0 ** -22 * (1 + np.abs(wlse))
        assert (np.abs(gl - wlse)[fin] <= ltol[fin]).all()


def run_attention(c, **kw):
    out, lse = sv.tree_attention(*c.args(), scale=c.scale, return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


ATTENTION = [
    dict(k=0, lens=(0, 1, 15, 16, 17)), dict(k=0, lens=(127, 128, 129, 300), hq=2, hkv=2),
    dict(k=5, lens=(37, 0, 130)), dict(k=5, lens=(37, 0, 130), dtype="f16"),
    dict(k=1, D=64, hq=3, hkv=1, lens=(5, 200)), dict(k=7, D=64, dtype="f16", page=8, lens=(31, 32, 33, 95)),
    dict(k=7, D=96, page=32, lens=(100, 3)), dict(k=16, D=96, dtype="f16", hq=10, hkv=2, page=4, lens=(61, 128)),
    dict(k=3, D=256, page=64, lens=(70, 500)), dict(k=16, D=256, dtype="f16", hq=16, hkv=2, lens=(33, 127)),
    dict(k=16, hq=16, hkv=2, lens=(255, 600), page=128), dict(k=64, hq=8, hkv=1, lens=(40, 700), page=16),
    dict(k=64, hq=2, hkv=2, D=64, lens=(1, 2, 3), page=1), dict(k=64, hq=4, hkv=2, D=256, lens=(64, 65), page=1024),
    dict(k=8, hq=14, hkv=2, lens=(77, 1000, 5), absent=0.4), dict(k=64, hq=5, hkv=1, lens=(20,), absent=0.2),
    dict(k=64, hq=256, hkv=1, D=64, lens=(50,)), dict(k=20, hq=256, hkv=2, D=256, lens=(9, 70)),
    dict(k=4, lens=(10, -1, 0, -5, 60), absent=0.3), dict(k=2, lens=(-1, -1)),
    dict(k=6, lens=(50, 90), amp=8.0), dict(k=6, lens=(50, 90), amp=8.0, dtype="f16", D=64),
    dict(k=6, lens=(50, 90), fill=float("inf")), dict(k=6, lens=(50, 90), scale=1e-3),
]


@pytest.mark.parametrize("kw", ATTENTION, ids=lambda kw: "-".join("%s%s" % i for i in kw.items()).replace(" ", ""))
def test_attention(dev, kw):
    print("attention", kw, flush=True)
    c = Case(dev, **kw)
    c.check(*run_attention(c))


def test_attention_many_sequences(dev):
    """More sequences than one scan step, most of them short, one long: the shares cross many units."""
    rs = np.random.RandomState(3)
    lens = [int(n) for n in rs.randint(-1, 40, 333)]
    lens[200] = 3000
    c = Case(dev, k=2, hq=2, hkv=1, D=64, lens=tuple(lens), absent=0.1)
    c.check(*run_attention(c))


def test_attention_strided_queries_and_offsets(dev):
    """Queries out of a joint projection, and of a transposed layout."""
    c = Case(dev, k=4, hq=8, hkv=2, lens=(40, 9))
    q, *rest = c.args()
    joint = torch.full((2, 5, 12, 128), float("nan"), dtype=q.dtype, device=dev)
    joint[:, :, 1:9] = q
    out, lse = sv.tree_attention(joint[:, :, 1:9], *rest, return_lse=True)
    c.check(out, lse)
    heads_first = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    out2, _ = sv.tree_attention(heads_first, *rest)
    assert torch.equal(out, out2)


def test_attention_value_nan_reaches_only_rows_that_see_it(dev):
    c = Case(dev, k=9, hq=8, hkv=2, lens=(70, 13))
    c.parents[:] = np.array([-1, -1, 0, 0, 1, 1, 2, 4, 4], np.int32)
    see = ref.sees(c.parents[0], 9)
    clean = c.vc.clone()
    want, _ = run_attention(c)
    for b, n in enumerate((70, 13)):  # node 1 (row 2): one NaN and one infinity in its value
        pos = n + 2
        c.vc[c.table[b, pos // 16], :, pos % 16, 5] = float("nan")
        c.vc[c.table[b, pos // 16], :, pos % 16, 77] = float("inf")
    got, _ = run_attention(c)
    c.vc = clean
    for r in range(10):
        if see[r, 2]:
            assert torch.isnan(got[:, r, :, 5]).all() and torch.isinf(got[:, r, :, 77]).all()
            keep = [d for d in range(128) if d not in (5, 77)]
            assert torch.equal(got[:, r][..., keep], want[:, r][..., keep])
        else:
            assert torch.equal(got[:, r], want[:, r])


@pytest.mark.parametrize("pos", [0, 63, 69])
def test_attention_value_nan_of_a_committed_key_reaches_every_row(dev, pos):
    c = Case(dev, k=9, hq=8, hkv=2, lens=(70,), fill=0.0)
    want, _ = run_attention(c)
    c.vc[c.table[0, pos // 16], 1, pos % 16, 9] = float("nan")
    got, _ = run_attention(c)
    assert torch.isnan(got[0, :, 4:, 9]).all()
    keep = [d for d in range(128) if d != 9]
    assert torch.equal(got[..., keep], want[..., keep]) and torch.equal(got[:, :, :4], want[:, :, :4])


def test_attention_is_reproducible_and_leaves_inputs(dev):
    c = Case(dev, k=16, hq=16, hkv=2, lens=(900, 33, 2000), fill=0.0)
    a = c.args()
    before = [x.clone() for x in a]
    o1 = sv.tree_attention(*a, return_lse=True)
    o2 = sv.tree_attention(*a, return_lse=True)
    assert torch.equal(o1.out, o2.out) and torch.equal(o1.lse, o2.lse)
    assert all(torch.equal(x, y) for x, y in zip(before, a))


def test_attention_far_pages(dev):
    """Rows whose offset in the cache passes 2^32 elements (2^33 bytes)."""
    P, hkv, page, D = 4200, 32, 256, 128  # 4.4e9 elements
    kc = torch.empty((P, hkv, page, D), dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    c = Case(dev, k=3, hq=32, hkv=32, D=128, page=256, lens=(300, 70), fill=0.0)
    ids = np.array([[4199, 1], [4100, 0]], np.int32)
    for b in range(2):
        for s in range(c.table.shape[1]):
            if c.table[b, s] >= 0:
                kc[ids[b, s]] = c.kc[c.table[b, s]].to(dev)
                vc[ids[b, s]] = c.vc[c.table[b, s]].to(dev)
    q, _, _, _, lens, par = c.args()
    c.check(*sv.tree_attention(q, kc, vc, torch.from_numpy(ids).to(dev), lens, par, return_lse=True))


def test_attention_pages_out_of_range_stay_in_bounds(dev):
    """Page numbers of -1 and beyond the cache under attended positions: the other sequence is not touched."""
    c = Case(dev, k=2, lens=(40, 40), fill=0.0)
    good = run_attention(c)[0]
    c.table[0, 0], c.table[0, 1] = -1, 1 << 30
    got = run_attention(c)[0]
    assert torch.equal(got[1], good[1])


def test_attention_too_long_for_the_table_is_absent(dev):
    c = Case(dev, k=2, lens=(40, 20), fill=0.0)
    c.lens[0] = c.table.shape[1] * 16 - 2
    out, lse = run_attention(c)
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    assert torch.isfinite(lse[1]).all()


def test_attention_graph_follows_lengths_and_trees(dev):
    c = Case(dev, k=4, lens=(40, 90), fill=0.0)
    q, kc, vc, table, lens, par = c.args()
    other = torch.tensor([7, 80], dtype=torch.int32, device=dev)
    flat = torch.full_like(par, -1)
    eager = []
    for n, p in ((lens, par), (other, flat)):
        eager.append(sv.tree_attention(q, kc, vc, table, n.clone(), p.clone(), return_lse=True))
    cur_n, cur_p = lens.clone(), par.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        sv.tree_attention(q, kc, vc, table, cur_n, cur_p, return_lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = sv.tree_attention(q, kc, vc, table, cur_n, cur_p, return_lse=True)
    for turn in range(6):
        cur_n.copy_((lens, other)[turn % 2])
        cur_p.copy_((par, flat)[turn % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res.out, eager[turn % 2].out) and torch.equal(res.lse, eager[turn % 2].lse)
        sv.tree_attention(q, kc, vc, table, cur_n, cur_p)  # eager work between replays


# ------------------------------------------------------------------------------------------------------- the walk

def logits_case(seed, B, k, V, T, onehot, dtype="f32", width=3, gap=0.7, absent=0.1):
    rs = np.random.RandomState(seed)
    t = torch.from_numpy(rs.randn(B, k + 1, V) * 2).to(DT[dtype])
    par = np.full((B, k), -2, np.int32)
    for b in range(B):
        kids = {}
        for i in range(k):
            if rs.rand() < absent:
                continue
            ok = [p for p in range(max(-1, i - 8), i) if (p < 0 or par[b, p] != -2) and kids.get(p, 0) < width]
            if ok:
                par[b, i] = ok[rs.randint(len(ok))]
                kids[par[b, i]] = kids.get(par[b, i], 0) + 1
    R = int(par.max()) + 2
    d = (t[:, :R].double() + gap * torch.from_numpy(rs.randn(B, R, V))).to(DT[dtype])
    tok = np.zeros((B, k), np.int32)
    for b in range(B):
        for i in range(k):
            if par[b, i] == -2:
                tok[b, i] = rs.randint(-5, V + 5)
                continue
            row = (t if onehot or T == 0 else d)[b, par[b, i] + 1].double().numpy() / (T or 1.0)
            p = np.exp(row - row.max())
            tok[b, i] = np.argmax(row) if rs.rand() < 0.4 else rs.choice(V, p=p / p.sum())
    return t, d, tok, par, rs.rand(B, k + 1).astype(np.float32)


def check_walk(dev, t, d, tok, par, u, T, onehot):
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    r = sv.verify_tree(on(t), None if d is None else on(d), on(tok), on(par), on(u), T, onehot=onehot)
    torch.cuda.synchronize()
    acc, out, path = (x.cpu().numpy() for x in r)
    t64 = t.double().numpy()
    d64 = None if d is None else d.double().numpy()
    depth = []
    for b in range(len(tok)):
        a, o, p, margin = ref.walk(t64[b], None if d64 is None or onehot else d64[b], tok[b], par[b],
                                   u[b].astype(np.float64), T, onehot)
        if margin <= 1.0:  # closer to a border than the kernel's sums tell apart
            continue
        assert (acc[b], list(out[b]), list(path[b])) == (a, o, p), "sequence %d" % b
        depth.append(a)
    return depth


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
@pytest.mark.parametrize("T", [0.0, 0.6, 1.0, 2.5])
@pytest.mark.parametrize("B,k,V", [(9, 4, 1000), (5, 16, 4099), (3, 64, 333), (7, 1, 1), (6, 5, 2), (4, 9, 8192), (2, 20, 40000)])
def test_walk(dev, dtype, onehot, T, B, k, V):
    print("walk", dtype, onehot, T, B, k, V, flush=True)
    check_walk(dev, *logits_case(B * 100 + k, B, k, V, T, onehot, dtype), T, onehot)


@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
@pytest.mark.parametrize("B", [1, 40, 300])
def test_walk_large_vocabulary(dev, onehot, B):
    """The vocabulary of the verification workloads, rows of one likely token over a Gaussian tail."""
    V, k = 151936 if B < 300 else 20011, 6
    g = torch.Generator(device=dev).manual_seed(B)
    t = torch.randn((B, k + 1, V), device=dev, generator=g) * 2
    top = torch.randint(0, V, (B, k + 1, 1), device=dev, generator=g)
    t.scatter_(2, top, torch.logsumexp(t, 2, keepdim=True))
    t = t.to(torch.bfloat16)
    par = np.tile(np.array([-1, -1, 0, 0, 1, 2], np.int32), (B, 1))
    d = (t[:, :4].float() + 0.5 * torch.randn((B, 4, V), device=dev, generator=g)).to(torch.bfloat16)
    if onehot:
        tok = np.ascontiguousarray(top[:, :, 0].cpu().numpy()[np.arange(B)[:, None], par + 1].astype(np.int32))
        tok[:, [0, 3]] = (tok[:, [0, 3]] + 1) % V
    else:
        pick = torch.multinomial(torch.softmax(d.float().view(-1, V), 1), 2, replacement=True, generator=g).view(B, 4, 2)
        tok = np.ascontiguousarray(pick.cpu().numpy()[:, [0, 0, 1, 1, 2, 3], [0, 1, 0, 1, 0, 0]].astype(np.int32))
    u = torch.rand((B, k + 1), device=dev, generator=g).cpu().numpy()
    some = list(range(0, B, max(1, B // 20)))
    r = sv.verify_tree(t, d, torch.from_numpy(tok).to(dev), torch.from_numpy(par).to(dev), torch.from_numpy(u).to(dev),
                       1.0, onehot=onehot)
    acc, out, path = (x.cpu().numpy() for x in r)
    ts, ds = t[some].double().cpu().numpy(), d[some].double().cpu().numpy()
    for i, b in enumerate(some):
        a, o, p, margin = ref.walk(ts[i], ds[i], tok[b], par[b], u[b].astype(np.float64), 1.0, onehot)
        if margin > 1.0:
            assert (acc[b], list(out[b]), list(path[b])) == (a, o, p), "sequence %d" % b


def test_walk_on_a_chain_is_verify(dev):
    """parents i - 1: the same accepted lengths and tokens as sv_verify (whose sums are 32-bit; these uniforms stand off
    the borders by more than 1e-5, checked by the reference's margin)."""
    B, k, V = 12, 6, 1000
    rs = np.random.RandomState(5)
    t = torch.from_numpy(rs.randn(B, k + 1, V) * 2).float()
    d = (t[:, :k].double() + 0.4 * torch.from_numpy(rs.randn(B, k, V))).float()
    p = torch.softmax(d.double(), -1).numpy()
    tok = np.array([[rs.choice(V, p=p[b, i] / p[b, i].sum()) for i in range(k)] for b in range(B)], np.int32)
    u = rs.rand(B, k + 1).astype(np.float32)
    par = np.tile(np.arange(-1, k - 1, dtype=np.int32), (B, 1))
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    for onehot in (False, True):
        a = sv.verify(on(t), on(d), on(tok), on(u), 1.0, onehot=onehot)
        r = sv.verify_tree(on(t), on(d), on(tok), on(par), on(u), 1.0, onehot=onehot)
        for b in range(B):
            margin = ref.walk(t[b].double().numpy(), d[b].double().numpy(), tok[b], par[b], u[b].astype(np.float64), 1.0,
                              onehot, e=1e-5)[3]
            if margin > 1.0:
                assert int(a.accepted_len[b]) == int(r.accepted_len[b])
                assert torch.equal(a.out_tokens[b], r.out_tokens[b])


@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
@pytest.mark.parametrize("T,amp,shift", [(1e-4, 1.0, 0.0), (0.05, 30.0, 0.0), (50.0, 300.0, -2e4), (1.0, 1.0, 1e6), (1.0, 200.0, 0.0)])
def test_walk_extreme_temperatures_and_logits(dev, T, amp, shift, onehot):
    """Rows that are one token, rows that are flat, and logits far from zero: l / T from 1e-2 to 1e6."""
    t, d, tok, par, u = logits_case(8, 12, 10, 6000, 1.0, onehot, absent=0.0)
    t, d = t * amp + shift, d * amp + shift
    for b in range(12):
        for i in range(10):
            if (b + i) % 2:
                tok[b, i] = int(t[b, par[b, i] + 1].argmax())
    check_walk(dev, t, d, tok, par, u, T, onehot)


def test_walk_refused_trees(dev):
    B, k, V = 8, 4, 50
    t, d, tok, par, u = logits_case(1, B, k, V, 1.0, False, absent=0.0)
    par[:] = np.array([-1, 0, 0, 1], np.int32)
    tok %= V
    d = t[:, :3].clone()
    par[0, 2] = 2      # itself
    par[1, 1] = 3      # a later node
    par[2, 0] = -3
    par[3, 1] = -2     # node 3 hangs on an absent one
    tok[4, 3] = V
    tok[5, 0] = -1
    par[6, 3] = 2      # row 3 of the draft is not there
    depth = check_walk(dev, t, d, tok, par, u, 1.0, False)
    assert depth[:7] == [-1] * 7 and depth[7] >= 0


def test_walk_ties_masked_tokens_and_extreme_uniforms(dev):
    B, k, V = 6, 3, 700
    t = torch.zeros(B, k + 1, V)
    t[:, :, ::2] = -float("inf")  # masked tokens are never drawn
    par = np.tile(np.array([-1, -1, 0], np.int32), (B, 1))
    tok = np.tile(np.array([1, 3, 5], np.int32), (B, 1))
    u = np.zeros((B, k + 1), np.float32)
    u[0] = 1 - 2.0 ** -24
    u[1] = 0.0
    u[2:] = np.random.RandomState(0).rand(B - 2, k + 1)
    for onehot in (True, False):
        check_walk(dev, t, t[:, :2].clone(), tok, par, u, 1.0, onehot)
    check_walk(dev, t, None, tok, par, u, 0.0, True)


def test_walk_first_token_distribution(dev):
    """Losslessness: the first committed token over many independent trees follows the target's p (chi-square; 13 cells,
    12 degrees of freedom, 99.99% quantile 39.1)."""
    V, N = 13, 60000
    rs = np.random.RandomState(11)
    p = rs.rand(V) ** 2 + 0.02
    q = rs.rand(V) ** 2 + 0.02
    p, q = p / p.sum(), q / q.sum()
    par = np.tile(np.array([-1, -1, -1], np.int32), (N, 1))
    tok = rs.choice(V, size=(N, 3), p=q).astype(np.int32)
    t = torch.from_numpy(np.log(p)).float().to(dev).expand(N, 4, V).contiguous()
    d = torch.from_numpy(np.log(q)).float().to(dev).expand(N, 1, V).contiguous()
    on = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    for onehot in (False, True):
        u = rs.rand(N, 4).astype(np.float32)
        first = sv.verify_tree(t, d, on(tok), on(par), on(u), 1.0, onehot=onehot).out_tokens[:, 0].cpu().numpy()
        got = np.bincount(first, minlength=V)
        assert ((got - N * p) ** 2 / (N * p)).sum() < 39.1


def test_walk_repeats_on_one_workspace_and_in_a_graph(dev):
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    t, d, tok, par, u = (on(x) for x in logits_case(4, 20, 12, 5000, 1.0, False))
    first = [x.clone() for x in sv.verify_tree(t, d, tok, par, u, 1.0)]
    u2 = torch.rand_like(u)
    second = [x.clone() for x in sv.verify_tree(t, d, tok, par, u2, 1.0)]
    cur = u.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r = sv.verify_tree(t, d, tok, par, cur, 1.0)
    for turn in range(6):
        cur.copy_((u, u2)[turn % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, (first, second)[turn % 2]))
        sv.verify_tree(t, d, tok, par, u, 1.0)


def test_walk_calls_of_other_shapes_on_one_workspace(dev):
    """A workspace serves calls of any shape in turn: small and large batches, every row at once and rows read as the walk
    comes to them, one and several workgroups per row."""
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    shapes = [(1, 20, 9000, False), (60, 6, 5000, False), (3, 4, 40, True), (2, 30, 30000, True), (90, 3, 9000, False),
              (1, 2, 100000, False), (300, 2, 4500, True)]
    for i, (B, k, V, onehot) in enumerate(shapes + shapes):
        t, d, tok, par, u = logits_case(i, B, k, V, 1.0, onehot)
        args = (on(t), None if onehot else on(d), on(tok), on(par), on(u), 1.0)
        want = sv.verify_tree(*args, onehot=onehot, workspace=torch.zeros(1 << 24, dtype=torch.uint8, device=dev))
        got = sv.verify_tree(*args, onehot=onehot, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (B, k, V, onehot)
        assert int(got.accepted_len.min()) >= 0


@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
@pytest.mark.parametrize("T", [0.0, 1.0])
def test_walk_when_no_workgroup_waits(dev, onehot, T):
    """The longest wait set to nothing: workgroups leave before the others' parts are there, and the walks are ended by
    the kernel that follows, with the same results; the workspace serves the next call as ever."""
    import ctypes

    lib = sv.load_library()
    lib.sv_internal_tree_wait.argtypes = [ctypes.c_uint64]
    cases = [logits_case(B, B, k, V, T, onehot) for B, k, V in ((40, 12, 30000), (3, 20, 9000), (100, 5, 20000))]
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    args = [tuple(on(x) for x in c) for c in cases]
    want = [[x.clone() for x in sv.verify_tree(*a, T, onehot=onehot)] for a in args]
    try:
        for ticks in (0, 200):
            lib.sv_internal_tree_wait(ticks)
            for a, w in zip(args, want):
                got = sv.verify_tree(*a, T, onehot=onehot)
                torch.cuda.synchronize()
                assert all(torch.equal(x, y) for x, y in zip(got, w))
    finally:
        lib.sv_internal_tree_wait(2000000)
    for a, w in zip(args, want):
        assert all(torch.equal(x, y) for x, y in zip(sv.verify_tree(*a, T, onehot=onehot), w))


@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
def test_walk_when_some_workgroups_leave(dev, onehot):
    """Waits of about as long as a pass takes: a workgroup may leave, the first one too, in a pass in which the others
    see a node kept and the token drawn."""
    import ctypes

    lib = sv.load_library()
    lib.sv_internal_tree_wait.argtypes = [ctypes.c_uint64]
    cases = [logits_case(B, B, k, V, 1.0, onehot) for B, k, V in ((90, 6, 20000), (100, 5, 20000), (60, 16, 50000))]
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    args = [tuple(on(x) for x in c) for c in cases]
    want = [[x.clone() for x in sv.verify_tree(*a, 1.0, onehot=onehot)] for a in args]
    try:
        for ticks in (30, 60, 100, 150, 220, 300, 500) * 3:
            lib.sv_internal_tree_wait(ticks)
            for i, (a, w) in enumerate(zip(args, want)):
                got = sv.verify_tree(*a, 1.0, onehot=onehot)
                assert all(torch.equal(x, y) for x, y in zip(got, w)), (ticks, i)
    finally:
        lib.sv_internal_tree_wait(2000000)


def test_walks_on_two_streams_at_once(dev):
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    cases = [tuple(on(x) for x in logits_case(i, 120, 8, 40000, 1.0, False)) for i in range(2)]
    want = [[x.clone() for x in sv.verify_tree(*c, 1.0)] for c in cases]
    calls = [sv.TreeVerifier(*c, 1.0) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for call, st in zip(calls, streams):
            call(stream=st.cuda_stream)
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        got = (call.accepted_len, call.out_tokens, call.path)
        assert all(torch.equal(x, y) for x, y in zip(got, w))


# ------------------------------------------------------------------------------------------------------- the cache

def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("kw", [dict(t=1), dict(t=17, D=64, page=8), dict(t=40, D=96, hkv=1, page=4), dict(t=300, D=256, page=128),
                                dict(t=5, D=8, page=1)], ids=str)
def test_append(dev, kw):
    t, D, hkv, page = kw["t"], kw.get("D", 128), kw.get("hkv", 2), kw.get("page", 16)
    rs = np.random.RandomState(t)
    lens = np.array([0, 5, 33, -1, page * 2], np.int32)
    count = np.array([t, max(1, t // 2), 0, t, t + 9], np.int32)
    table, P = paged(rs, [max(0, n) + t for n in lens], page)
    table[4, -1] = -1  # the last page is missing: rows there are dropped
    kc = torch.randn((P, hkv, page, D)).to(torch.bfloat16)
    vc = torch.randn_like(kc)
    new = torch.randn((5, t, 2 * hkv + 1, D)).to(torch.bfloat16)
    kd, vd, nd = kc.to(dev), vc.to(dev), new.to(dev)
    sv.cache_append(nd[:, :, :hkv], nd[:, :, hkv + 1:], kd, vd, torch.from_numpy(table).to(dev),
                    torch.from_numpy(lens).to(dev), count=torch.from_numpy(count).to(dev))
    for b, n in enumerate(lens):
        for j in range(min(int(count[b]), t) if n >= 0 else 0):
            i = table[b, (n + j) // page]
            if i >= 0:
                kc[i, :, (n + j) % page] = new[b, j, :hkv]
                vc[i, :, (n + j) % page] = new[b, j, hkv + 1:]
    assert same_bits(kd.cpu(), kc) and same_bits(vd.cpu(), vc)


@pytest.mark.parametrize("k,layers,D,page", [(1, 1, 64, 16), (16, 3, 128, 8), (64, 2, 96, 32), (64, 1, 256, 1)])
def test_commit(dev, k, layers, D, page):
    rs = np.random.RandomState(k)
    lens = np.array([0, 7, 40, -1, 12, 30, 31, 9], np.int32)
    B = len(lens)
    acc = np.array([min(k, n) for n in (k, 0, k // 2, 1, -1, k // 3, k + 1, 2)], np.int32)
    acc[6] = k + 1
    path = np.full((B, k), -1, np.int32)
    for b in range(B):
        n = max(0, min(acc[b], k))
        path[b, :n] = np.sort(rs.permutation(k)[:n])
    if k > 2:
        path[7, :2] = [5, 5]  # not increasing: refused
    table, P = paged(rs, [max(0, n) + k + 1 for n in lens], page)
    kc = torch.randn((layers, P, 2, page, D)).to(torch.float16)
    vc = torch.randn_like(kc)
    kd, vd = kc.to(dev), vc.to(dev)
    on = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    n2 = sv.cache_commit(on(path), on(acc), kd, vd, on(table), on(lens)).cpu().numpy()
    for b, n in enumerate(lens):
        p = path[b, :max(0, acc[b])] if acc[b] <= k else []
        fine = n >= 0 and 0 <= acc[b] <= k and all(j <= p[j] < k for j in range(len(p))) and all(np.diff(p) > 0)
        assert n2[b] == (n + 1 + acc[b] if fine else n)
        for j in range(len(p) if fine else 0):
            a, z = n + 1 + p[j], n + 1 + j
            for c in (kc, vc):
                c[:, table[b, z // page], :, z % page] = c[:, table[b, a // page], :, a % page].clone()
    assert same_bits(kd.cpu(), kc) and same_bits(vd.cpu(), vc)


def books(rs, n, width, P, page, most):
    count = np.array([rs.randint(0, most + 1) for _ in range(n)], np.int32)
    order = list(rs.permutation(P))
    table, refs = np.full((n, width), -1, np.int32), np.zeros(P, np.int32)
    for b in range(n):
        for i in range(count[b]):
            if order and rs.rand() < 0.8:
                table[b, i] = order.pop()
            else:  # a shared page
                table[b, i] = rs.choice(np.nonzero(refs)[0]) if refs.any() else order.pop()
            refs[table[b, i]] += 1
    return table, count, refs


@pytest.mark.parametrize("n,width,P,page", [(1, 1, 1, 16), (5, 8, 30, 16), (40, 16, 200, 8), (300, 6, 9000, 1), (64, 300, 12000, 64),
                                            (4096, 3, 6000, 4)])
def test_resize(dev, n, width, P, page):
    rs = np.random.RandomState(n)
    table, count, refs = books(rs, n, width, P, page, min(width, max(1, P // n)))
    on = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    dt, dc, dr = on(table), on(count), on(refs)
    for turn in range(4):
        want = np.array([rs.choice([-1, 0, rs.randint(0, width * page + 1), rs.randint(0, width * page + 1)])
                         for _ in range(n)], np.int32)
        if turn == 2 and n > 3:
            want[3] = width * page + 1  # more than the table holds
        ok = sv.cache_resize(on(want), dt, dc, dr, page_size=page)
        status = ref.resize(want, table, count, refs, page)
        assert np.array_equal(ok.cpu().numpy(), status)
        assert np.array_equal(dt.cpu().numpy(), table)
        assert np.array_equal(dc.cpu().numpy(), count) and np.array_equal(dr.cpu().numpy(), refs)


@pytest.mark.parametrize("P_free", [0, 3, 50])
def test_fork(dev, P_free):
    page, layers = 8, 3
    rs = np.random.RandomState(P_free)
    n = 14
    lens = np.array([20, 16, 0, 7, 3] + [5] * 9, np.int32)
    table, P = paged(rs, [20, 16, 0, 7, 0] + [0] * 9, page, spare=P_free, width=4)
    count = (table >= 0).sum(1).astype(np.int32)
    refs = np.zeros(P, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    # slot 4 has more positions than pages; slot 5 twice; slot 3 is not empty; 99 and -1 do not exist; 6 from itself
    src = np.array([0, 1, 2, 3, 0, 4, 0, 99, 0, 6, 0, 11, 3], np.int32)
    dst = np.array([5, 7, 8, 9, 5, 10, 3, 10, -1, 6, 11, 12, 13], np.int32)
    kc = torch.randn((layers, P, 2, page, 64)).to(torch.bfloat16)
    vc = torch.randn_like(kc)
    kd, vd = kc.to(dev), vc.to(dev)
    on = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    dt, dc, dr, dl = on(table), on(count), on(refs), on(lens)
    status = sv.cache_fork(on(src), on(dst), kd, vd, dt, dc, dr, dl)
    want = ref.fork(src, dst, kc, vc, table, count, refs, lens, page)
    assert np.array_equal(status.cpu().numpy(), want)
    for a, b in ((dt, table), (dc, count), (dr, refs), (dl, lens)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert same_bits(kd.cpu(), kc) and same_bits(vd.cpu(), vc)


def test_cache_far_offsets(dev):
    """Positions whose offset in the cache passes 2^32 elements: append, commit and fork against plain indexing."""
    L, P, hkv, page, D = 2, 4200, 16, 256, 128  # 4.4e9 elements, the second layer's from 2.2e9 on
    kc = torch.empty((L, P, hkv, page, D), dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    table = torch.tensor([[4199, 4198], [-1, -1]], dtype=torch.int32, device=dev)
    count = torch.tensor([2, 0], dtype=torch.int32, device=dev)
    refs = torch.ones(P, dtype=torch.int32, device=dev)
    refs[4197] = 0
    lens = torch.tensor([250, 0], dtype=torch.int32, device=dev)
    new = torch.randn((L, 2, 9, 2, hkv, D), device=dev).to(torch.bfloat16)
    for l in range(L):
        sv.cache_append(new[l, :, :, 0], new[l, :, :, 1], kc[l], vc[l], table, lens)
    at = [(4199, 250 + j) if j < 6 else (4198, j - 6) for j in range(9)]
    for j, (i, o) in enumerate(at):
        assert torch.equal(kc[:, i, :, o], new[:, 0, j, 0]) and torch.equal(vc[:, i, :, o], new[:, 0, j, 1])
    path = torch.tensor([[1, 4, 7, -1, -1, -1, -1, -1], [-1] * 8], dtype=torch.int32, device=dev)
    acc = torch.tensor([3, -1], dtype=torch.int32, device=dev)
    n = sv.cache_commit(path, acc, kc, vc, table, lens)
    assert n.tolist() == [254, 0]
    for j, src in enumerate((1, 4, 7)):
        i, o = at[1 + j]
        assert torch.equal(kc[:, i, :, o], new[:, 0, 1 + src, 0]) and torch.equal(vc[:, i, :, o], new[:, 0, 1 + src, 1])
    ok = sv.cache_fork(torch.zeros(1, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev), kc, vc,
                       table, count, refs, n)
    assert ok.tolist() == [1] and table.tolist() == [[4199, 4198], [4197, -1]]
    assert torch.equal(kc[:, 4197, :, 250:254], kc[:, 4199, :, 250:254]) and torch.equal(vc[1, 4197, 3, 253], vc[1, 4199, 3, 253])


def test_resize_wishes_past_32_bits(dev):
    """Wishes that add up to more than 2^31 pages: the first sequence is served, the others are refused and unchanged."""
    width, P = 1 << 29, 64
    table = torch.full((6, width), -1, dtype=torch.int32, device=dev)
    count, refs = torch.zeros(6, dtype=torch.int32, device=dev), torch.zeros(P, dtype=torch.int32, device=dev)
    want = torch.tensor([10] + [width] * 4 + [5], dtype=torch.int32, device=dev)
    status = sv.cache_resize(want, table, count, refs, page_size=1)
    assert status.tolist() == [1, 0, 0, 0, 0, 0] and count.tolist() == [10, 0, 0, 0, 0, 0]
    assert refs.tolist() == [1] * 10 + [0] * (P - 10)
    assert table[:, :80].cpu().tolist() == [list(range(10)) + [-1] * 70] + [[-1] * 80] * 5
    want[1:] = torch.tensor([width] * 5, dtype=torch.int32, device=dev)  # 10 + 5 * 2^29 passes 2^31
    status = sv.cache_resize(want, table, count, refs, page_size=1)
    assert status.tolist() == [1, 0, 0, 0, 0, 0] and count.tolist() == [10, 0, 0, 0, 0, 0]
    assert refs.tolist() == [1] * 10 + [0] * (P - 10) and (table[1:, :80] == -1).all()


def test_empty_batches(dev):
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device=dev)
    out = sv.tree_attention(z(0, 4, 8, 64, t=torch.bfloat16), c, c.clone(), z(0, 3), z(0), z(0, 3), return_lse=True)
    assert out.out.shape == (0, 4, 8, 64) and out.lse.shape == (0, 4, 8)
    r = sv.verify_tree(z(0, 4, 10, t=torch.float32), None, z(0, 3), z(0, 3), None, 0.0)
    assert r.path.shape == (0, 3)
    sv.cache_append(z(0, 4, 2, 64, t=torch.bfloat16), z(0, 4, 2, 64, t=torch.bfloat16), c, c.clone(), z(0, 3), z(0))
    sv.cache_append(z(2, 0, 2, 64, t=torch.bfloat16), z(2, 0, 2, 64, t=torch.bfloat16), c, c.clone(), z(2, 3), z(2))
    k5 = c[None].contiguous()
    assert sv.cache_commit(z(0, 3), z(0), k5, k5.clone(), z(0, 3), z(0)).shape == (0,)
    assert sv.cache_fork(z(0), z(0), k5, k5.clone(), z(2, 3), z(2), z(4), z(2)).shape == (0,)
    assert sv.cache_resize(z(0), z(0, 3), z(0), z(4), page_size=16).shape == (0,)


# ------------------------------------------------------------------------------------------- a run of them together

def test_decode_steps_with_trees(dev):
    """Prompts in two layers' caches, groups forked, three steps of append, attention, walk, commit and resize; each
    step's attention and cache against the references, and one step as a graph against the eager one."""
    rs = np.random.RandomState(0)
    B, k, hkv, hq, D, page, layers, V = 6, 5, 2, 4, 64, 8, 2, 97
    P, width = 80, 12
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    kc, vc = (torch.zeros((layers, P, hkv, page, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
    table, count, refs, lens = i32(B, width) - 1, i32(B), i32(P), i32(B)
    prompt = np.array([13, 24, 0, 0, 0, 0], np.int32)
    assert sv.cache_resize(on(prompt), table, count, refs, page_size=page).all()
    kv = torch.randn((layers, B, 24, 2 * hkv, D)).to(torch.bfloat16).to(dev)
    for l in range(layers):
        sv.cache_append(kv[l, :, :, :hkv], kv[l, :, :, hkv:], kc[l], vc[l], table, lens, count=on(prompt))
    lens.copy_(on(prompt))
    assert sv.cache_fork(on(np.array([0, 0, 1, 1], np.int32)), on(np.array([2, 3, 4, 5], np.int32)), kc, vc, table, count, refs, lens).all()
    rows = {b: [(l, b0, j) for j in range(prompt[b0])] for b, b0 in enumerate([0, 1, 0, 0, 1, 1]) for l in [0]}
    hist = {b: [kv[:, b0, j].cpu() for j in range(prompt[b0])] for b, b0 in enumerate([0, 1, 0, 0, 1, 1])}
    par = on(np.tile(np.array([-1, -1, 0, 1, 2], np.int32), (B, 1)))
    for step in range(3):
        assert sv.cache_resize(lens + k + 1, table, count, refs, page_size=page).all()
        new = torch.randn((layers, B, k + 1, 2 * hkv, D)).to(torch.bfloat16).to(dev)
        q = torch.randn((B, k + 1, hq, D)).to(torch.bfloat16).to(dev)
        target = (torch.randn((B, k + 1, V)) * 2).to(dev)
        tok = torch.stack([target[b, par[b].long() + 1].argmax(1) for b in range(B)]).int()
        u = torch.rand((B, k + 1)).to(dev)

        def one():
            for l in range(layers):
                sv.cache_append(new[l, :, :, :hkv], new[l, :, :, hkv:], kc[l], vc[l], table, lens)
            att = [sv.tree_attention(q, kc[l], vc[l], table, lens, par, return_lse=True) for l in range(layers)]
            r = sv.verify_tree(target, None, tok, par, u, 1.0, onehot=True)
            return att, r, sv.cache_commit(r.path, r.accepted_len, kc, vc, table, lens)

        if step == 1:  # the same step captured: nothing of it runs until it is replayed
            state = [x.clone() for x in (kc, vc)]
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                att, r, n2 = one()
            for _ in range(3):
                kc.copy_(state[0])
                vc.copy_(state[1])
                graph.replay()
                torch.cuda.synchronize()
            got = [x.clone() for x in (*r, n2, kc, vc)] + [a.out.clone() for a in att]
            kc.copy_(state[0])
            vc.copy_(state[1])
            att, r, n2 = one()
            assert all(torch.equal(a, b) for a, b in zip(got, [*r, n2, kc, vc] + [a.out for a in att]))
        else:
            att, r, n2 = one()
        acc, path = r.accepted_len.cpu().numpy(), r.path.cpu().numpy()
        c = Case.__new__(Case)
        c.q, c.k, c.dtype, c.scale, c.parents = q.cpu(), k, "bf16", D ** -0.5, par.cpu().numpy()
        for l in range(layers):
            # attention against the history and this step's rows, laid out flat
            L = max(len(h) for h in hist.values()) + k + 1
            K = np.zeros((B, hkv, L, D))
            Vv = np.zeros((B, hkv, L, D))
            for b in range(B):
                seq = [x[l] for x in hist[b]] + list(new[l, b].cpu())
                for j, x in enumerate(seq):
                    K[b, :, j], Vv[b, :, j] = x[:hkv].double().numpy(), x[hkv:].double().numpy()
            c.lens = np.array([len(hist[b]) for b in range(B)], np.int32)
            c.compare(att[l].out, att[l].lse, *ref.attention(c.q.double().numpy(), K, Vv, np.arange(B)[:, None], c.lens, c.parents, c.scale))
        for b in range(B):
            hist[b] += [new[:, b, 0].cpu()] + [new[:, b, 1 + path[b, j]].cpu() for j in range(acc[b])]
        lens.copy_(n2)
        assert lens.tolist() == [len(hist[b]) for b in range(B)]
        kh, vh, th = kc.cpu(), vc.cpu(), table.cpu()
        for b in range(B):
            for j, x in enumerate(hist[b]):
                i = int(th[b, j // page])
                assert torch.equal(kh[:, i, :, j % page], x[:, :hkv]) and torch.equal(vh[:, i, :, j % page], x[:, hkv:])
    assert sv.cache_resize(i32(B), table, count, refs, page_size=page).all()
    assert not refs.any() and not count.any() and (table == -1).all()


def test_calls_on_another_stream(dev):
    c = Case(dev, k=4, lens=(40, 200), fill=0.0)
    a = c.args()
    want = sv.tree_attention(*a).out
    call = sv.TreeAttention(*a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [sv.tree_attention(*a).out, call().out.clone()]
    side.synchronize()
    assert all(torch.equal(want, g) for g in got)


def test_prepared_calls_in_two_graphs(dev):
    """A step's attention and walk captured twice, each with prepared calls of its own, replayed in turn and at once on two
    streams, with eager calls of other shapes between."""
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    walks, attns, want = [], [], []
    for i in range(2):
        c = Case(dev, k=5, lens=(300, 17, 900), fill=0.0, seed=i)
        w = tuple(on(x) for x in logits_case(30 + i, 12, 6, 30000, 1.0, False))
        attns.append(sv.TreeAttention(*c.args()))
        walks.append(sv.TreeVerifier(*w, 1.0))
        want.append([x.clone() for x in (*sv.verify_tree(*w, 1.0), sv.tree_attention(*c.args()).out)])
        attns[i](), walks[i]()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*walks[i](), attns[i]().out))
        graphs.append(g)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(4):
        for o in outs:
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(sides[i] if turn % 2 else sides[0]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], want[i])), (turn, i)
        small = tuple(on(x) for x in logits_case(turn, 3, 4, 5000, 1.0, True))
        sv.verify_tree(*small, 1.0, onehot=True)


@pytest.mark.parametrize("onehot", [False, True], ids=["logits", "onehot"])
def test_walk_of_the_most_sequences(dev, onehot):
    B, k, V = 65535, 2, 11
    rs = np.random.RandomState(9)
    t, d = (torch.from_numpy(rs.randn(B, n, V)).float() for n in (k + 1, k))
    tok = rs.randint(0, V, (B, k)).astype(np.int32)
    par = np.tile(np.array([-1, 0], np.int32), (B, 1))
    u = rs.rand(B, k + 1).astype(np.float32)
    on = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev)  # noqa: E731
    r = [x.cpu().numpy() for x in sv.verify_tree(on(t), on(d), on(tok), on(par), on(u), 0.7, onehot=onehot)]
    for b in list(range(0, B, 997)) + [B - 1]:
        *want, margin = ref.walk(t[b].double().numpy(), None if onehot else d[b].double().numpy(), tok[b], par[b],
                                 u[b].astype(np.float64), float(np.float32(0.7)), onehot)
        if margin > 1.0:
            assert [r[0][b], list(r[1][b]), list(r[2][b])] == want, b
