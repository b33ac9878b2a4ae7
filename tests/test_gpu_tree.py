"""Attention of drafted tokens (pa_decode_tree) against the definition in 64 bits.

Tolerances, with w the exact softmax weights of a row and A = sum_j w_j |v_j|:
  - the output is rounded to bf16 once: 2^-8 of the value;
  - the weights enter the product as bf16: each is off by at most 2^-8 of itself, A * 2^-8 together;
  - a score is off by at most e = d * 2^-23 * max_j sum |q k_j| * scale (fp32 accumulation that may truncate), the
    exponential of it and of the maximum by 2 e + 2^-20 relative, in the weights and in their sum: A * (4 e + 2^-19).
"""
import numpy as np
import pytest

from tests.gpu_helpers import i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Case:
    """A batch of drafted trees over a paged cache; every value that no row may see is poisoned."""

    def __init__(self, lens, counts, Hq, Hkv, d, bs, *, seed=0, masks="tree", poison=float("nan"), gain=1.0, tail=0,
                 pad=0, extra_words=0):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.counts, self.Hq, self.Hkv, self.d, self.bs = list(lens), list(counts), Hq, Hkv, d, bs
        B, self.T = len(self.lens), sum(counts) + tail
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.max_nodes = max([1, *counts]) + 32 * extra_words
        self.max_len = max(self.lens)
        blocks = [-(-n // bs) for n in self.lens]
        nb = sum(blocks) + 3
        order = rng.permutation(nb)
        spare = order[sum(blocks):]
        wide = max([1, *blocks]) + pad
        self.tables = np.resize(spare, (B, wide)).copy()  # padding names poisoned blocks
        at = 0
        for b in range(B):
            self.tables[b, :blocks[b]] = order[at:at + blocks[b]]
            at += blocks[b]
        self.nb = nb

        def normal(*shape):
            return (torch.randn(shape, generator=g)).to(torch.bfloat16)

        k, v = normal(nb, Hkv, bs, d), normal(nb, Hkv, bs, d)
        used = torch.zeros(nb, bs, dtype=torch.bool)
        for b in range(B):
            for j in range(blocks[b]):
                used[self.tables[b, j], :min(bs, self.lens[b] - j * bs)] = True
        for pool in (k, v):
            pool.permute(0, 2, 1, 3)[~used] = poison
        qkv = normal(self.T, Hq + 2 * Hkv, d)
        qkv[:, :Hq] *= gain
        if tail:
            qkv[self.T - tail:] = poison
        self.q, self.kt, self.vt = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.k, self.v = k, v
        words = -(-self.max_nodes // 32)
        bits = np.zeros((self.T, words * 32), bool)
        for b in range(B):
            n, lo = counts[b], self.cu[b]
            for i in range(n):
                if masks == "tree":
                    p = int(rng.integers(-1, i)) if i else -1
                    if p >= 0:
                        bits[lo + i] = bits[lo + p]
                    bits[lo + i, i] = True
                elif masks == "chain":
                    bits[lo + i, :i + 1] = True
                elif masks == "random":
                    bits[lo + i, :n] = rng.random(n) < 0.5
                    bits[lo + i, n:] = rng.random(words * 32 - n) < 0.5  # past the tree: not looked at
        self.bits = bits
        self.masks = None if masks == "chain" else np.packbits(bits, axis=1, bitorder="little").view(np.int32)
        self.scale = float(np.float32(d ** -0.5))

    def launch(self, pt=0, *, stream=None, contiguous=False, fill=None, masks=True, workspace=None, max_len=None):
        import torch
        import paged_kv_cache_349_b200 as pa
        q, kt, vt = (x.contiguous().cuda() if contiguous else x for x in (self.q, self.kt, self.vt))
        if not contiguous:
            qkv = torch.cat([self.q, self.kt, self.vt], 1).cuda()
            q, kt, vt = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
        out = torch.full((self.T, self.Hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        L = self.max_len if max_len is None else max_len
        size = pa.pa_decode_tree_workspace_size(len(self.lens), self.T, self.Hq, self.Hkv, self.d, self.bs, L,
                                                self.max_nodes, pt)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        if ws is not None and fill is not None:
            ws.fill_(fill)
        pa.pa_decode_tree(out, q, kt, vt, self.k.cuda(), self.v.cuda(), i32_dev(self.tables), i32_dev(self.lens),
                          i32_dev(self.cu), None if self.masks is None else i32_dev(self.masks), max_seq_len=L,
                          max_nodes=self.max_nodes, scale=self.scale, partition_tokens=pt, workspace=ws, err_flag=flag)
        torch.cuda.synchronize()
        self.flag = int(flag.item())
        return out

    def rows(self, b):
        """Exact keys and values of sequence b in order: [L + n, Hkv, d]."""
        L, lo, n = self.lens[b], self.cu[b], self.counts[b]
        pages = self.tables[b, :-(-L // self.bs)]
        got = []
        for pool, tree in ((self.k, self.kt), (self.v, self.vt)):
            x = pool[pages].transpose(1, 2).reshape(-1, self.Hkv, self.d)[:L]
            got.append(np.concatenate([x.double().numpy(), tree[lo:lo + n].double().numpy()]))
        return got

    def exact(self, b):
        """(out, tolerance) of the rows of sequence b, [n, Hq, d]; what is not seen is left out altogether."""
        import warnings
        L, lo, n, G = self.lens[b], self.cu[b], self.counts[b], self.Hq // self.Hkv
        k, v = self.rows(b)
        q = self.q[lo:lo + n].double().numpy()
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        for i in range(n):
            seen = np.concatenate([np.ones(L, bool), self.bits[lo + i, :n]])
            if not seen.any():
                continue
            ks, vs = k[seen], v[seen]
            for h in range(self.Hkv):
                qs = q[i, h * G:(h + 1) * G]
                with warnings.catch_warnings():
                    warnings.simplefilter("ignore")
                    s = (ks[:, h] @ qs.T).T * self.scale
                    w = np.exp(s - s.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    A = w @ np.abs(vs[:, h])
                    o = w @ vs[:, h]
                    e = self.d * 2.0 ** -23 * (np.abs(ks[:, h]) @ np.abs(qs).T).max() * self.scale
                out[i, h * G:(h + 1) * G] = o
                tol[i, h * G:(h + 1) * G] = np.abs(o) * 2.0 ** -8 + A * (2.0 ** -8 + 4 * e + 2.0 ** -19)
        return out, tol

    def check(self, out, only=None):
        got = out.double().cpu().numpy()
        for b in range(len(self.lens)) if only is None else only:
            lo, hi = self.cu[b], self.cu[b + 1]
            want, tol = self.exact(b)
            x = got[lo:hi]
            assert np.array_equal(np.isfinite(want), np.isfinite(x)), f"sequence {b}"
            fine = np.isfinite(want)
            err = np.abs(x - want)
            assert (err[fine] <= tol[fine]).all(), f"sequence {b}: {np.max((err - tol)[fine])}"
        assert (got[self.cu[-1]:] == 7.0).all()  # rows behind the last sequence, left as they were


SHAPES = [(64, 8, 4, 2), (64, 16, 8, 1), (128, 16, 4, 4), (128, 32, 8, 2), (128, 64, 8, 8), (128, 8, 2, 1)]
LENS = [0, 1, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 391]


@pytest.mark.parametrize("d,bs,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("pt", [-1, 128, 0])
def test_ragged_lengths_and_trees(d, bs, Hq, Hkv, pt):
    counts = [1, 5, 0, 17, 2, 31, 32, 33, 1, 64, 3, 9, 12, 65]
    c = Case(LENS, counts, Hq, Hkv, d, bs, seed=d + bs + Hq, tail=3, pad=2)
    c.check(c.launch(pt))
    assert c.flag == 0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 32, 33, 64, 100, 129, 200])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (4, 2), (2, 2)])
def test_node_counts(n, Hq, Hkv):
    """Rows that fill a tile, spill into the next one, and trees over several tiles of keys."""
    c = Case([130, 0, 77], [n, max(1, n // 2), n], Hq, Hkv, 128, 16, seed=n)
    c.check(c.launch())
    assert c.flag == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("masks", ["chain", "random", "none"])
def test_other_masks(d, masks):
    """A chain without masks; any bits; no bits at all: rows without a cached token are zero then."""
    c = Case([0, 40, 256, 0], [70, 33, 5, 1], 4, 2, d, 16, seed=d, masks=masks, extra_words=1)
    out = c.launch()
    c.check(out)
    if masks == "none":
        assert not bool(out[:70].any()) and not bool(out[-1].any())


@pytest.mark.parametrize("poison", [float("inf"), -float("inf"), 3.0e38])
def test_poison_kinds(poison):
    c = Case([0, 3, 100, 190], [9, 6, 40, 20], 8, 2, 128, 32, seed=3, poison=poison, tail=5)
    c.check(c.launch())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_unseen_nodes_stay_out(d, bad, where):
    """NaN and infinities in nodes: they reach the rows that see the node, no others."""
    c = Case([37, 0, 150], [40, 70, 11], 4, 2, d, 16, seed=11)
    for b, nodes in ((0, [4, 39]), (1, [0, 33, 69]), (2, [10])):
        for i in nodes:
            (c.kt if where == "k" else c.vt)[c.cu[b] + i, 1, 3] = bad
    got = c.launch().double().cpu().numpy()
    for b in range(3):
        want, tol = c.exact(b)
        x = got[c.cu[b]:c.cu[b + 1]]
        sees = np.zeros(want.shape, bool)
        for i in range(c.counts[b]):
            mine = c.bits[c.cu[b] + i, :c.counts[b]]
            touched = [j for j in np.nonzero(mine)[0] if j in dict(((0, [4, 39]), (1, [0, 33, 69]), (2, [10])))[b]]
            if touched and where == "v":
                sees[i, 2:, 3] = True  # the heads of key head 1, that value alone
            elif touched:
                sees[i, 2:] = True
        assert np.isfinite(x[~sees]).all() and (np.abs(x - want)[~sees] <= tol[~sees]).all()
        if where == "v":  # a weight times the value, which is not finite whatever the weight
            assert np.array_equal(np.isnan(x[sees]), np.isnan(want[sees]))
            same = ~np.isnan(want[sees])
            assert np.array_equal(x[sees][same], want[sees][same])
        elif not bad < 0:  # a key of -inf may only lower the score; NaN and +inf scores spoil the row
            assert np.array_equal(np.isfinite(x[sees]), np.isfinite(want[sees]))


def test_attended_nan_of_the_cache_reaches_its_sequence_only():
    c = Case([40, 40], [5, 5], 4, 2, 128, 16, seed=2)
    c.v[c.tables[0, 1], 0, 3, 7] = float("nan")
    out = c.launch().float().cpu().numpy()
    assert np.isnan(out[:5, :2, 7]).all()
    out[:5, :2, 7] = 0
    assert np.isfinite(out).all()


def test_large_scores():
    """Scores of hundreds: the running maximum moves often and far."""
    for gain in (30.0, 1e-3):
        c = Case([300, 511, 64], [33, 8, 40], 8, 2, 128, 16, seed=5, gain=gain)
        c.check(c.launch())
        c.check(c.launch(128))


def test_rising_scores_move_the_maximum_every_tile():
    import torch
    c = Case([900], [20], 4, 1, 64, 16, seed=6)
    direction = torch.randn(64).to(torch.bfloat16)
    c.q[:] = direction
    for j in range(-(-900 // 16)):
        c.k[c.tables[0, j], 0] = (direction.float() * (j - 20) * 0.2).to(torch.bfloat16)
    c.k[c.tables[0, 56], 0, 4:] = float("nan")
    c.check(c.launch())


@pytest.mark.parametrize("pt", [128, 384, 0])
def test_split_over_a_long_cache(pt):
    c = Case([2500, 1, 2048, 129], [12, 40, 3, 7], 8, 2, 128, 16, seed=8)
    for fill in (0, 255):
        c.check(c.launch(pt, fill=fill))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,counts,Hq", [([9000], [3], 2), ([9000], [20], 8), ([5001, 3, 3000], [5, 1, 33], 8), ([4000], [0], 4),
                                            ([9000], [9], 8)])
def test_many_pieces_of_one_unit(d, lens, counts, Hq):
    """Few rows and a long cache: dozens of pieces to join, more than there are rows."""
    c = Case(lens, counts, Hq, 1, d, 16, seed=d + Hq, tail=2)
    for fill in (0, 255):
        c.check(c.launch(128, fill=fill))
        assert c.flag == 0


def test_results_do_not_depend_on_placement_or_neighbours():
    """Bit-identical when blocks move and when a sequence runs alone."""
    import torch
    c = Case([200, 77, 500], [9, 30, 64], 8, 2, 128, 32, seed=9)
    first = c.launch(-1)
    assert torch.equal(first, c.launch(-1, contiguous=True))
    perm = torch.from_numpy(np.random.default_rng(1).permutation(c.nb))
    k, v = torch.empty_like(c.k), torch.empty_like(c.v)
    k[perm], v[perm] = c.k, c.v
    c.k, c.v, c.tables = k, v, perm.numpy()[c.tables]
    assert torch.equal(first, c.launch(-1))
    alone = Case([500], [64], 8, 2, 128, 32, seed=0)
    lo = c.cu[2]
    alone.q, alone.kt, alone.vt, alone.k, alone.v = c.q[lo:], c.kt[lo:], c.vt[lo:], c.k, c.v
    alone.tables, alone.masks, alone.nb = c.tables[2:], c.masks[lo:], c.nb
    assert torch.equal(first[lo:], alone.launch(-1))


def test_flags():
    import paged_kv_cache_349_b200 as pa
    c = Case([64, 70, 33], [4, 4, 4], 4, 2, 128, 16, seed=4)
    kept = c.tables[1, 1]
    for bad in (-1, c.nb, 2 ** 31 - 1):
        c.tables[1, 1] = bad
        out = c.launch()
        assert c.flag == pa.PA_FLAG_BAD_BLOCK
        c.check(out, only=[0, 2])
    # the tokens of the block are left out: as a sequence without them
    short = Case([54], [4], 4, 2, 128, 16, seed=0)
    t = c.tables[1]
    short.tables = np.array([[t[0], t[2], t[3], t[4], 0]])
    short.k, short.v, short.nb = c.k, c.v, c.nb
    short.q, short.kt, short.vt, short.bits = c.q[4:8], c.kt[4:8], c.vt[4:8], c.bits[4:8]
    want, tol = short.exact(0)
    assert (np.abs(out[4:8].double().cpu().numpy() - want) <= tol).all()
    c.tables[1, 1] = kept
    c.lens = [64, -3, 33]
    out = c.launch(max_len=64)
    assert c.flag == pa.PA_FLAG_BAD_LEN
    c.lens[1] = 0
    c.check(out)
    c.lens = [64, 70, 33]
    out = c.launch(max_len=64)  # longer than the caller said: cut
    assert c.flag == pa.PA_FLAG_BAD_LEN
    c.lens[1] = 64
    c.check(out)
    # more nodes than the caller said, and bounds outside of the rows
    c = Case([20, 20], [3, 9], 4, 2, 64, 16, seed=4, masks="chain")
    c.max_nodes = 5
    out = c.launch()
    assert c.flag == pa.PA_FLAG_BAD_LEN
    assert bool((out[8:] == 7.0).all())
    c.counts, c.cu = [3, 5], np.array([0, 3, 8])
    c.check(out[:8])
    c = Case([20, 20], [3, 3], 4, 2, 64, 16, seed=4, masks="chain")
    c.cu = np.array([-4, 3, 11])
    out = c.launch()
    assert c.flag == pa.PA_FLAG_BAD_LEN
    c.cu = np.array([0, 3, 6])
    c.check(out)


def test_streams_graphs_and_a_shared_workspace():
    """On a side stream, captured, replayed after the inputs changed, and two graphs on one workspace in turn."""
    import torch
    import paged_kv_cache_349_b200 as pa
    cases = [Case([700, 300], [16, 9], 8, 2, 128, 16, seed=s) for s in (1, 2)]
    want = [c.launch(128) for c in cases]
    size = max(pa.pa_decode_tree_workspace_size(2, c.T, 8, 2, 128, 16, 700, 16, 128) for c in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs, outs, state = [], [], []
    side = torch.cuda.Stream()
    for c in cases:
        dev = [x.contiguous().cuda() for x in (c.q, c.kt, c.vt, c.k, c.v)] + [i32_dev(x) for x in
                                                                             (c.tables, c.lens, c.cu, c.masks)]
        out = torch.empty(c.T, 8, 128, dtype=torch.bfloat16, device="cuda")
        call = lambda: pa.pa_decode_tree(out, *dev, max_seq_len=700, max_nodes=16, scale=c.scale, partition_tokens=128,
                                         workspace=ws)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append(out)
        state.append(dev)
    for _ in range(3):
        for g, out, w in zip(graphs, outs, want):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    state[0][6].copy_(i32_dev([650, 5]))  # other lengths in the same graph
    graphs[0].replay()
    torch.cuda.synchronize()
    cases[0].lens = [650, 5]
    cases[0].check(outs[0])


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 2), (64, 8, 1), (128, 4, 1)])
@pytest.mark.parametrize("pt", [-1, 128, 0])
def test_trees_of_one_and_of_two_row_groups_in_turn(d, Hq, Hkv, pt):
    """Trees whose rows fill one group of 128, two of them or several pairs follow each other on one SM."""
    c = Case([300, 1200, 77, 900, 640, 64, 2000, 0, 513], [33, 3, 40, 0, 17, 64, 1, 16, 48], Hq, Hkv, d, 16, seed=d + Hq,
             tail=1)
    c.check(c.launch(pt, fill=255))
    assert c.flag == 0


def test_two_row_groups_for_trees_of_one():
    """max_nodes calls for two groups of rows, no tree has more than one; a width of masks beyond every tree."""
    c = Case([700, 130, 1, 64], [5, 16, 1, 9], 8, 1, 128, 16, seed=12, extra_words=3)
    c.check(c.launch(128))
    assert c.flag == 0


def test_more_sequences_than_threads():
    rng = np.random.default_rng(5)
    c = Case(rng.integers(0, 90, 1203), rng.integers(0, 3, 1203), 4, 2, 64, 8, seed=5)
    c.check(c.launch(-1))
    c.check(c.launch(128, max_len=600))  # room for cuts, of which each unit is too short
    assert c.flag == 0


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own, while both are at work."""
    import torch
    import paged_kv_cache_349_b200 as pa
    cases = [Case([3000, 900], [16, 9], 8, 2, 128, 16, seed=1), Case([2500, 1800], [64, 30], 8, 1, 128, 16, seed=2)]
    want = [c.launch(128) for c in cases]
    jobs = []
    for c in cases:
        dev = [x.contiguous().cuda() for x in (c.q, c.kt, c.vt, c.k, c.v)] + [i32_dev(x) for x in
                                                                             (c.tables, c.lens, c.cu, c.masks)]
        size = pa.pa_decode_tree_workspace_size(2, c.T, c.Hq, c.Hkv, 128, 16, c.max_len, c.max_nodes, 128)
        jobs.append((c, dev, torch.empty(size, dtype=torch.uint8, device="cuda"),
                     [torch.empty(c.T, c.Hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(20)],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(20):
        for c, dev, ws, outs, stream in jobs:
            pa.pa_decode_tree(outs[i], *dev, max_seq_len=c.max_len, max_nodes=c.max_nodes, scale=c.scale,
                              partition_tokens=128, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for (c, dev, ws, outs, stream), w in zip(jobs, want):
        assert all(torch.equal(o, w) for o in outs)


def test_pool_offsets_past_32_bits():
    """Blocks at the end of pools of more than 2^31 values, read here and written by pa_rope_and_cache."""
    import torch
    import paged_kv_cache_349_b200 as pa
    c = Case([300, 45], [9, 4], 16, 8, 128, 16, seed=3)
    small = c.launch(128)
    total = 2 ** 31 // (8 * 16 * 128) + 64
    pools = [torch.empty(total, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for pool, part in zip(pools, (c.k, c.v)):
        pool[total - c.nb:] = part.cuda()
    tables = i32_dev(c.tables + (total - c.nb))
    size = pa.pa_decode_tree_workspace_size(2, c.T, 16, 8, 128, 16, c.max_len, c.max_nodes, 128)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty(c.T, 16, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_tree(out, c.q.contiguous().cuda(), c.kt.contiguous().cuda(), c.vt.contiguous().cuda(), *pools, tables,
                      i32_dev(c.lens), i32_dev(c.cu), i32_dev(c.masks), max_seq_len=c.max_len, max_nodes=c.max_nodes,
                      scale=c.scale, partition_tokens=128, workspace=ws)
    assert torch.equal(out, small)
    k, v = c.kt.contiguous().cuda(), c.vt.contiguous().cuda()
    slots = torch.arange(total * 16 - c.T, total * 16, dtype=torch.int32, device="cuda")
    turns, _ = pa.pa_rope_frequencies(128)
    pa.pa_rope_and_cache(None, None, k, v, *pools, slots, torch.zeros_like(slots), turns.cuda())  # position 0: no turn
    for pool, rows in zip(pools, (k, v)):
        assert torch.equal(pool[-2:].transpose(1, 2).reshape(32, 8, 128)[32 - c.T:], rows)


def test_python_refusals():
    import torch
    import paged_kv_cache_349_b200 as pa
    c = Case([20], [3], 4, 2, 64, 16, seed=4)
    dev = [x.contiguous().cuda() for x in (c.q, c.kt, c.vt, c.k, c.v)] + [i32_dev(x) for x in
                                                                         (c.tables, c.lens, c.cu, c.masks)]
    out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    kw = dict(max_seq_len=20, max_nodes=3, scale=0.1)
    pa.pa_decode_tree(out, *dev, **kw)

    def put(i, x):
        return [*dev[:i], x, *dev[i + 1:]]

    for args, k in ((put(1, dev[1][:2]), kw), (put(7, dev[7][:1]), kw), (put(5, dev[5].view(-1)), kw),
                    (dev, dict(kw, max_nodes=40)), (put(0, dev[0].transpose(0, 1).contiguous().transpose(0, 1)), kw)):
        with pytest.raises(ValueError):
            pa.pa_decode_tree(out, *args, **k)
    for args in (put(0, dev[0].float()), put(3, dev[3].float()), put(6, dev[6].long()), put(4, dev[4].cpu())):
        with pytest.raises(TypeError):
            pa.pa_decode_tree(out, *args, **kw)
    with pytest.raises(pa.PaError):
        pa.pa_decode_tree(out, *dev, **dict(kw, partition_tokens=100))


@pytest.mark.parametrize("Hq,Hkv,extra", [(4, 2, 0), (8, 1, 2)])
@pytest.mark.parametrize("pt", [-1, 128])
def test_bounds_that_decrease(Hq, Hkv, extra, pt):
    """Every row has one owner: a sequence that begins below an earlier bound has no nodes, the others keep theirs."""
    import paged_kv_cache_349_b200 as pa
    c = Case([900, 37, 1300, 700], [5, 3, 6, 6], Hq, Hkv, 64, 16, seed=4, masks="chain", extra_words=extra)
    c.max_nodes = max(c.max_nodes, 9)
    c.bits[:9] = np.arange(c.bits.shape[1]) <= np.arange(9)[:, None]
    c.cu = np.array([0, 9, 5, 14, 20])  # rows 9..13 are nobody's
    out = c.launch(pt)
    assert c.flag == pa.PA_FLAG_BAD_LEN
    assert bool((out[9:14] == 7.0).all())
    c.counts, c.cu = [9, 0, 0, 6], np.array([0, 9, 9, 14, 20])
    c.check(out, only=[0, 3])


def test_a_bound_beyond_those_of_many_sequences():
    """More sequences than threads: one bound that is too large takes the rows of all sequences below it."""
    import paged_kv_cache_349_b200 as pa
    B = 700
    c = Case(np.random.default_rng(6).integers(0, 200, B), [1] * B, 4, 2, 64, 8, seed=6, masks="chain")
    c.cu[3] = 600
    for pt in (-1, 128):
        out = c.launch(pt, max_len=600)
        assert c.flag == pa.PA_FLAG_BAD_LEN
        assert bool((out[3:600] == 7.0).all())
        c.cu[3] = 3
        c.check(out, only=[0, 1, 2, *range(600, B)])
        c.cu[3] = 600


@pytest.mark.parametrize("nodes,Hq,Hkv,d,extra", [(5, 8, 2, 128, 0), (9, 8, 2, 64, 0), (30, 8, 2, 128, 0), (3, 4, 4, 128, 0),
                                                   (7, 16, 2, 128, 2), (17, 8, 1, 64, 0)])
def test_uncut_results_do_not_depend_on_neighbours(nodes, Hq, Hkv, d, extra):
    """The rows behind a tree's last node hold the next sequence's queries, or none: whatever their scores are, the
    tree's own rows keep their bits.  Gain 30 makes the neighbour's maximum rise by dozens in tile after tile."""
    import torch
    neighbours = [700, 333]
    c = Case([900, *neighbours], [nodes, 6, 16], Hq, Hkv, d, 16, seed=nodes, extra_words=extra, tail=2, poison=0.0)
    quiet = c.launch(-1)
    c.check(quiet)
    for gain in (30.0, -200.0, float("nan"), float("inf")):
        q = c.q.clone()
        c.q[nodes:] *= gain
        loud = c.launch(-1)
        assert torch.equal(loud[:nodes], quiet[:nodes]), gain
        c.q[:] = q
    alone = Case([900], [nodes], Hq, Hkv, d, 16, seed=0)
    alone.q, alone.kt, alone.vt, alone.k, alone.v = c.q[:nodes], c.kt[:nodes], c.vt[:nodes], c.k, c.v
    alone.tables, alone.nb = c.tables[:1], c.nb
    for most in (c.max_nodes, nodes):  # one or two groups of rows in a CTA
        alone.max_nodes = most
        alone.masks = np.ascontiguousarray(c.masks[:nodes, :-(-most // 32)])
        assert torch.equal(alone.launch(-1), quiet[:nodes]), most


@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-40, 1e-38, 1.7e-38, 1e-30])
@pytest.mark.parametrize("pt", [-1, 128])
def test_scales_of_nothing(scale, pt):
    """Down to the smallest fp32 and 0: all weights are the same, and what a row does not see stays out."""
    for Hq, Hkv in ((4, 2), (8, 1)):
        c = Case([0, 1, 300, 777], [5, 3, 40, 20], Hq, Hkv, 64, 16, seed=9)
        c.scale = float(np.float32(scale))
        c.check(c.launch(pt))
    c = Case([0, 1, 300, 777], [5, 3, 40, 20], 4, 2, 64, 16, seed=9, gain=1e36)  # scores of up to 1e38
    c.scale = float(np.float32(scale))
    if scale < 1e-29:
        c.check(c.launch(pt))


@pytest.mark.parametrize("scale", [1.0, 1e6, 1e8, 1e12, 1e30, 2.3e38])
@pytest.mark.parametrize("pt", [-1, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1)])
def test_scales_up_to_the_largest(scale, pt, Hq, Hkv):
    """Scaled scores far beyond 2^30 and beyond fp32: a row is the mean of the values at its largest score.

    Every key is 1, 2 or 3 in all dimensions and q is 1, -1, 0 or 2^-7, so that scores are exact and other scores are at
    least 2^-1 scale below, or (q = 0) the same.  The mean's weights are all alike: 2^-8 of it for their rounding, which
    their sum does not have, 2^-8 for the output's, 2^-13 for fp32 sums of 1000 terms.  Where scale is 1 the others have
    weights: the definition's own tolerance.
    """
    import torch
    c = Case([700, 0, 300, 65], [12, 3, 40, 1], Hq, Hkv, 64, 16, seed=3, masks="chain", poison=0.0)
    c.scale = float(np.float32(scale))
    rng = np.random.default_rng(1)
    for keys in (c.k, c.kt):
        a = torch.from_numpy(rng.integers(1, 4, keys.shape[:-1])).to(torch.bfloat16)
        keys[:] = a[..., None]
    for h in range(Hq):
        c.q[:, h] = (1.0, -1.0, 0.0, 2.0 ** -7)[h % 4]
    out = c.launch(pt, fill=255)
    assert c.flag == 0
    if scale == 1.0:
        return c.check(out)
    got = out.double().cpu().numpy()
    for b in range(4):
        k, v = (x[:, 0] for x in c.rows(b))
        for i in range(c.counts[b]):
            seen = np.concatenate([np.ones(c.lens[b], bool), c.bits[c.cu[b] + i, :c.counts[b]]])
            for h in range(Hq):
                score = k[seen] @ c.q[c.cu[b] + i, h].double().numpy()
                best = v[seen][score == score.max()]
                want, A = best.mean(0), np.abs(best).mean(0)
                err = np.abs(got[c.cu[b] + i, h] - want)
                assert (err <= np.abs(want) * 2.0 ** -8 + A * (2.0 ** -8 + 2.0 ** -13)).all(), (b, i, h)
