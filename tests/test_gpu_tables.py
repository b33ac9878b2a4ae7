"""Tables, slots and masks built on the device, against plain Python; whole numbers have to be equal."""
import numpy as np
import pytest

from tests.gpu_helpers import i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def host(t):
    return t.cpu().numpy()


def model(tables, lens, add, free, cursor, bs, rows, cu_rows=None, path=None):
    """What the call should leave behind: tables, lens, cursor, slots, positions, cu_tokens, flag."""
    import paged_kv_cache_349_b200 as pa
    tables, flag = tables.copy(), 0
    B, mb = tables.shape
    n = []
    for L, a in zip(lens, add):
        ok = L >= 0 and a >= 0 and L + a <= mb * bs and (path is None or a <= path.shape[1])
        flag |= 0 if ok else pa.PA_FLAG_BAD_LEN
        n.append(int(a) if ok else 0)
    need = [max(0, -(-(L + a) // bs) - -(-L // bs)) if a else 0 for L, a in zip(lens, n)]
    bad = 0
    if cursor < 0 or cursor + sum(need) > len(free):
        bad |= pa.PA_FLAG_NO_BLOCKS
    if path is None and sum(n) > rows:
        bad |= pa.PA_FLAG_BAD_LEN
    slots, pos = np.full(rows, -1), np.zeros(rows, int)
    if bad:
        return tables, lens, cursor, slots, pos, np.zeros(B + 1, int), flag | bad
    cu = np.concatenate([[0], np.cumsum(n)])
    for b in range(B):
        have = -(-lens[b] // bs)
        tables[b, have:have + need[b]] = free[cursor:cursor + need[b]] if need[b] else []
        cursor += need[b]
        named = set()
        for k in range(n[b]):
            r = cu[b] + k if path is None else cu_rows[b] + path[b, k]
            if path is not None and (path[b, k] in named or not 0 <= path[b, k] < cu_rows[b + 1] - cu_rows[b]):
                continue
            named.add(path[b, k] if path is not None else k)
            at = lens[b] + k
            slots[r], pos[r] = tables[b, at // bs] * bs + at % bs, at
    return tables, np.asarray(lens) + n, cursor, slots, pos, cu, flag


def run(tables, lens, add, free, cursor, bs, rows, num_blocks, cu_rows=None, path=None, in_place=True, positions=True):
    import torch
    import paged_kv_cache_349_b200 as pa
    t, L, c = i32_dev(tables), i32_dev(lens), i32_dev([cursor])
    slots = torch.full((rows,), 7777, dtype=torch.int32, device="cuda")
    pos = torch.full((rows,), 7777, dtype=torch.int32, device="cuda") if positions else None
    cu = torch.full((len(lens) + 1,), 7777, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    Lo, co = (L, c) if in_place else (torch.empty_like(L), torch.empty_like(c))
    pa.pa_extend_tables(t, L, i32_dev(add), i32_dev(free), c, num_blocks=num_blocks, block_size=bs, slot_mapping=slots,
                        cu_tokens=cu, positions=pos, seq_lens_out=Lo, cursor_out=co,
                        cu_rows=None if path is None else i32_dev(cu_rows), path=None if path is None else i32_dev(path),
                        err_flag=flag)
    if not in_place:
        assert np.array_equal(host(L), lens) and host(c)[0] == cursor
    return host(t), host(Lo), int(host(co)[0]), host(slots), host(pos) if positions else None, host(cu), int(flag.item())


def same(got, want):
    for name, g, w in zip(("tables", "lens", "cursor", "slots", "positions", "cu_tokens", "flag"), got, want):
        if g is not None:
            assert np.array_equal(g, w), name


def batch(rng, lens, bs, extra, spare):
    """Tables of the given lengths with room for `extra` tokens each, and the free list behind them."""
    lens = np.asarray(lens)
    have = -(-lens // bs)
    mb = int((-(-(lens + extra) // bs)).max()) + 1
    order = rng.permutation(int((-(-(lens + extra) // bs)).sum()) + spare)
    tables, at = np.full((len(lens), mb), -9), 0
    for b, n in enumerate(have):
        tables[b, :n] = order[at:at + n]
        at += n
    return tables, order[at:], len(order)


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("B,hi,most", [(1, 0, 1), (1, 40, 300), (5, 33, 3), (64, 300, 130), (1024, 50, 2), (2500, 20, 9)])
def test_packed(bs, B, hi, most):
    rng = np.random.default_rng(B + bs)
    lens, add = rng.integers(0, hi + 1, size=B), rng.integers(0, most + 1, size=B)
    tables, free, nb = batch(rng, lens, bs, add, 4)
    for rows in (int(add.sum()), int(add.sum()) + 11):
        want = model(tables, lens, add, free, 0, bs, rows)
        same(run(tables, lens, add, free, 0, bs, rows, nb), want)
        same(run(tables, lens, add, np.concatenate([[-5, -5], free]), 2, bs, rows, nb, in_place=False, positions=False),
             (*want[:2], want[2] + 2, *want[3:]))


def test_prompts_of_a_whole_batch():
    """Tables from the lengths alone, more rows than the planning CTA maps itself."""
    rng = np.random.default_rng(3)
    add = rng.integers(1, 3000, size=41)
    lens = np.zeros(41, int)
    tables, free, nb = batch(rng, lens, 16, add, 0)
    same(run(tables, lens, add, free, 0, 16, int(add.sum()) + 3, nb), model(tables, lens, add, free, 0, 16, int(add.sum()) + 3))


@pytest.mark.parametrize("B,nodes,most", [(1, 1, 1), (7, 5, 5), (256, 33, 6), (200, 64, 8)])
def test_path_of_drafted_trees(B, nodes, most):
    rng = np.random.default_rng(B)
    bs = 16
    lens, add = rng.integers(0, 400, size=B), rng.integers(0, most + 1, size=B)
    counts = rng.integers(most, nodes + 1, size=B)
    cu = np.concatenate([[0], np.cumsum(counts)])
    path = np.full((B, most), -1)
    for b in range(B):
        path[b, :add[b]] = np.sort(rng.permutation(counts[b])[:add[b]])
    tables, free, nb = batch(rng, lens, bs, add, 1)
    rows = int(cu[-1]) + 2
    same(run(tables, lens, add, free, 0, bs, rows, nb, cu, path), model(tables, lens, add, free, 0, bs, rows, cu, path))


def test_odd_paths():
    """A node named twice counts where it is named first; names outside the tree and unused entries name nothing."""
    bs, lens, add = 8, [7, 3, 0], [4, 2, 0]
    path = np.array([[2, 2, 5, 0], [9, 1, 0, 0], [0, 1, 2, 0]])
    cu = np.array([1, 7, 10, 13])  # row 0 belongs to nobody
    rng = np.random.default_rng(0)
    tables, free, nb = batch(rng, lens, bs, np.asarray(add), 2)
    same(run(tables, lens, add, free, 0, bs, 15, nb, cu, path), model(tables, lens, add, free, 0, bs, 15, cu, path))
    add = [4, 5, 0]  # more than the path holds: that sequence gets no token
    same(run(tables, lens, add, free, 0, bs, 15, nb, cu, path), model(tables, lens, add, free, 0, bs, 15, cu, path))


def test_all_or_nothing_and_bad_lengths():
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(5)
    lens, add = np.array([10, 0, 33, 16]), np.array([30, 5, 1, 17])
    tables, free, nb = batch(rng, lens, 16, add, 0)
    need = model(tables, lens, add, free, 0, 16, 60)[2]
    for case in ((free[:need - 1], 0, 60), (free, 1 + len(free) - need, 60), (free, -1, 60), (free, 0, 52)):
        want = model(tables, lens, add, *case[:2], 16, case[2])
        assert want[-1] in (pa.PA_FLAG_NO_BLOCKS, pa.PA_FLAG_BAD_LEN) and (want[3] == -1).all()
        same(run(tables, lens, add, *case[:2], 16, case[2], nb), want)
    for L, a in (([10, -1, 33, 16], add), (lens, [30, -5, 1, 17]), (lens, [30, 5, 10 ** 6, 17]),
                 ([10, 2 ** 31 - 1, 33, 16], add)):
        want = model(tables, np.asarray(L), np.asarray(a), free, 0, 16, 60)
        assert want[-1] == pa.PA_FLAG_BAD_LEN
        same(run(tables, L, a, free, 0, 16, 60, nb), want)


def test_bad_block_ids_give_no_slot():
    import paged_kv_cache_349_b200 as pa
    tables = np.array([[3, -9, -9], [99, -9, -9]])
    got = run(tables, [14, 3], [4, 2], [50, 4], 0, 16, 6, 10)  # ids 99 and 50 are outside the pool of 10
    assert got[-1] == pa.PA_FLAG_BAD_BLOCK
    assert got[3].tolist() == [3 * 16 + 14, 3 * 16 + 15, -1, -1, -1, -1]
    assert got[4].tolist() == [14, 15, 16, 17, 3, 4]
    assert got[0].tolist() == [[3, 50, -9], [99, -9, -9]]


def test_steps_follow_each_other_and_replay():
    """Captured once and replayed: each replay continues from the lengths and the cursor the last one left."""
    import torch
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(8)
    B, bs, steps = 9, 8, 12
    lens = rng.integers(0, 20, size=B)
    tables, free, nb = batch(rng, lens, bs, 3 * steps, 0)
    t, L, f, c = i32_dev(tables), i32_dev(lens), i32_dev(free), i32_dev([0])
    add, slots, cu = i32_dev(np.zeros(B)), i32_dev(np.zeros(3 * B)), i32_dev(np.zeros(B + 1))
    call = lambda: pa.pa_extend_tables(t, L, add, f, c, num_blocks=nb, block_size=bs, slot_mapping=slots, cu_tokens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    state, cursor = tables, 0
    for _ in range(steps):
        a = rng.integers(0, 4, size=B)
        add.copy_(i32_dev(a))
        graph.replay()
        state, lens, cursor, want, _, wcu, _ = model(state, lens, a, free, cursor, bs, 3 * B)
        assert np.array_equal(host(t), state) and np.array_equal(host(L), lens) and host(c)[0] == cursor
        assert np.array_equal(host(slots), want) and np.array_equal(host(cu), wcu)


def tree(rng, n, width):
    return [max(-1, i - 1 - int(rng.integers(0, width))) if rng.random() > 0.2 else -1 for i in range(n)]


def masks_model(parents, cu, lens, rows, max_nodes):
    words = -(-max_nodes // 32)
    masks, pos = np.zeros((rows, words), np.uint32), np.zeros(rows, int)
    for b in range(len(lens)):
        for i in range(min(cu[b + 1] - cu[b], max_nodes)):
            j, depth = i, -1
            while j >= 0:
                masks[cu[b] + i, j // 32] |= np.uint32(1 << (j % 32))
                depth += 1
                p = parents[cu[b] + j]
                j = p if -1 <= p < j else -1
            pos[cu[b] + i] = lens[b] + depth
    return masks.view(np.int32), pos


@pytest.mark.parametrize("counts,max_nodes,width", [([1], 1, 1), ([8, 0, 3, 31, 32, 33], 33, 4), ([512, 1, 300], 512, 2),
                                                    ([64] * 100, 64, 20), ([7, 5], 200, 3), ([500], 512, 1)])
def test_tree_masks(counts, max_nodes, width):
    import torch
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(sum(counts))
    parents = np.array([p for n in counts for p in tree(rng, n, width)] + [3, 3])
    if width == 1:
        parents[1:counts[0]] = np.arange(counts[0] - 1)  # a chain
    cu, lens = np.concatenate([[0], np.cumsum(counts)]), rng.integers(0, 10000, size=len(counts))
    rows = len(parents)  # two rows belong to no sequence
    masks = torch.full((rows, -(-max_nodes // 32)), -1, dtype=torch.int32, device="cuda")
    pos, flag = i32_dev(np.full(rows, 9)), i32_dev([0])
    pa.pa_tree_masks(masks, pos, i32_dev(parents), i32_dev(cu), i32_dev(lens), max_nodes=max_nodes, err_flag=flag)
    want, wpos = masks_model(parents, cu, lens, rows, max_nodes)
    assert np.array_equal(host(masks), want) and np.array_equal(host(pos), wpos) and int(flag.item()) == 0
    masks.fill_(-1)
    pa.pa_tree_masks(masks, None, i32_dev(parents), i32_dev(cu), i32_dev(lens), max_nodes=max_nodes)
    assert np.array_equal(host(masks), want)


@pytest.mark.parametrize("cu,parents,max_nodes,flag", [
    ([0, 3, 6], [0, -1, 5, -2, 0, 1], 4, "BAD_TREE"),      # own number, a later node, below -1
    ([0, 5, 6], [-1, 0, 1, 2, 3, -1], 3, "BAD_LEN"),        # more nodes than max_nodes
    ([-2, 3, 99], [-1, 0, 1, -1, 0, 1], 4, "BAD_LEN"),      # bounds outside of the rows
    ([4, 2, 6], [-1, 0, -1, 0, 0, 1], 4, "BAD_LEN"),        # bounds that decrease
])
def test_tree_masks_bad_input(cu, parents, max_nodes, flag):
    import torch
    import paged_kv_cache_349_b200 as pa
    T = len(parents)
    masks, pos, f = torch.full((T, 1), -1, dtype=torch.int32, device="cuda"), i32_dev(np.full(T, 9)), i32_dev([0])
    pa.pa_tree_masks(masks, pos, i32_dev(parents), i32_dev(cu), i32_dev([10, 20]), max_nodes=max_nodes, err_flag=f)
    assert int(f.item()) == getattr(pa, "PA_FLAG_" + flag)
    if flag == "BAD_TREE":
        assert host(masks)[:, 0].tolist() == [1, 2, 4, 1, 3, 7] and host(pos).tolist() == [10, 10, 10, 20, 21, 22]
    elif cu == [0, 5, 6]:
        assert host(masks)[:, 0].tolist() == [1, 3, 7, 0, 0, 1] and host(pos).tolist() == [10, 11, 12, 0, 0, 20]
    elif cu[0] == -2:
        assert host(masks)[:, 0].tolist() == [1, 3, 7, 1, 3, 7] and host(pos).tolist() == [10, 11, 12, 20, 21, 22]


@pytest.mark.parametrize("cu,bits,positions", [
    ([4, 2, 6], [0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0]),
    ([0, 5, 3, 8], [1, 3, 7, 15, 31, 0, 0, 0], [10, 11, 12, 13, 14, 0, 0, 0]),
    ([2, 4, 1, 3, 4, 7], [0, 0, 1, 3, 1, 3, 7], [0, 0, 10, 11, 50, 51, 52]),
    ([6, 6, 0, 6], [0] * 6, [0] * 6),
])
def test_tree_masks_bounds_that_decrease(cu, bits, positions):
    """Every row has one owner: a sequence that begins below an earlier bound has no nodes."""
    import torch
    import paged_kv_cache_349_b200 as pa
    T, B = len(bits), len(cu) - 1
    parents = [x.bit_length() - 2 if x else -1 for x in bits]  # chains
    for _ in range(20):
        masks, pos, flag = torch.full((T, 1), -1, dtype=torch.int32, device="cuda"), i32_dev(np.full(T, 9)), i32_dev([0])
        pa.pa_tree_masks(masks, pos, i32_dev(parents), i32_dev(cu), i32_dev(10 * np.arange(1, B + 1)), max_nodes=8,
                         err_flag=flag)
        assert int(flag.item()) == pa.PA_FLAG_BAD_LEN
        assert host(masks)[:, 0].tolist() == bits and host(pos).tolist() == positions


def test_tree_masks_of_more_sequences_than_threads():
    """One early bound that is too large takes the rows of all sequences below it, of none above."""
    import torch
    import paged_kv_cache_349_b200 as pa
    B = 700
    cu = np.arange(B + 1)
    cu[3] = 600
    masks, pos, flag = torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), i32_dev(np.full(B, 9)), i32_dev([0])
    pa.pa_tree_masks(masks, pos, i32_dev(np.full(B, -1)), i32_dev(cu), i32_dev(np.arange(B)), max_nodes=1, err_flag=flag)
    want, wpos = np.ones(B, int), np.arange(B)
    want[3:600] = wpos[3:600] = 0  # row 2 is the first node of the sequence that ends at 600
    assert int(flag.item()) == pa.PA_FLAG_BAD_LEN
    assert np.array_equal(host(masks)[:, 0], want) and np.array_equal(host(pos), wpos)


@pytest.mark.parametrize("bad", [-1, -2 ** 31])
def test_paths_that_end_early(bad):
    """A negative entry among the accepted ones: that sequence gets no token and is flagged, the others get theirs."""
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(1)
    bs, lens, add = 8, np.array([7, 3, 0, 30]), np.array([3, 2, 4, 1])
    cu = np.array([0, 6, 9, 14, 20])
    whole = np.array([[0, 2, 5, -1], [0, 1, -1, -1], [0, 1, 3, 4], [2, -1, -1, -1]])
    tables, free, nb = batch(rng, lens, bs, add, 2)
    for b, k in ((0, 0), (0, 2), (1, 1), (2, 3), (3, 0)):
        path, kept = whole.copy(), add.copy()
        path[b, k], kept[b] = bad, 0
        want = model(tables, lens, kept, free, 0, bs, 20, cu, whole)
        same(run(tables, lens, add, free, 0, bs, 20, nb, cu, path), (*want[:-1], pa.PA_FLAG_BAD_LEN))
    same(run(tables, lens, add, free, 0, bs, 20, nb, cu, whole), model(tables, lens, add, free, 0, bs, 20, cu, whole))


@pytest.mark.parametrize("cu", [[0, 9, 6, 14], [-1, 6, 9, 14], [0, 6, 9, 21], [3, 1, 9, 14], [0, 6, 9, 2 ** 31 - 1]])
def test_bounds_of_drafted_rows(cu):
    """Bounds that decrease or leave the rows: nothing changes, no row gets a slot."""
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(2)
    lens, add = np.array([7, 3, 0]), np.array([3, 2, 4])
    path = np.array([[0, 2, 5, -1], [0, 1, -1, -1], [0, 1, 3, 4]])
    tables, free, nb = batch(rng, lens, 8, add, 2)
    for in_place in (True, False):
        got = run(tables, lens, add, free, 0, 8, 20, nb, np.array(cu), path, in_place=in_place)
        same(got, (tables, lens, 0, np.full(20, -1), np.zeros(20), np.zeros(4), pa.PA_FLAG_BAD_LEN))


@pytest.mark.parametrize("B,n", [(2367, 2), (2368, 2), (5000, 3), (20000, 1)])
def test_tree_masks_of_many_sequences(B, n):
    """More sequences than CTAs, in order and with a bound that is too large among the sequences of one CTA."""
    import torch
    import paged_kv_cache_349_b200 as pa
    cu, lens, rows = np.arange(B + 1) * n, np.arange(B), B * n + 1
    parents = np.append(np.tile(np.arange(n) - 1, B), 7)  # chains; the last row is nobody's
    masks, pos, flag = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda"), i32_dev(np.full(rows, 9)), i32_dev([0])
    want, wpos = masks_model(parents, cu, lens, rows, n)
    pa.pa_tree_masks(masks, pos, i32_dev(parents), i32_dev(cu), i32_dev(lens), max_nodes=n, err_flag=flag)
    assert np.array_equal(host(masks), want) and np.array_equal(host(pos), wpos) and int(flag.item()) == 0
    at, to = B // 3, B // 3 + 50
    cu[at] = to * n  # sequence at - 1 reaches up to sequence `to`, with n nodes at most; those between have none
    want[at * n:to * n] = wpos[at * n:to * n] = 0
    masks.fill_(-1)
    pa.pa_tree_masks(masks, pos, i32_dev(parents), i32_dev(cu), i32_dev(lens), max_nodes=n, err_flag=flag)
    assert np.array_equal(host(masks), want) and np.array_equal(host(pos), wpos)
    assert int(flag.item()) == pa.PA_FLAG_BAD_LEN
