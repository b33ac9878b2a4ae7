"""The drafting calls together, as a serving loop uses them: masks, rotary positions, attention of the drafted
tokens, table growth and the cache write of the accepted path -- captured once and replayed step after step.

The oracle keeps every sequence's accepted tokens as plain lists of 64-bit rows.  The tree attention has to match
the definition over them, and at the end pa_decode over the cache that the steps built has to match it too.
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


def attend(q, k, v, scale):
    """Weights and A = sum w |v| as in the tree attention's own test."""
    s = k @ q * scale
    w = np.exp(s - s.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v), len(q) * 2.0 ** -23 * (np.abs(k) @ np.abs(q)).max() * scale


@pytest.mark.parametrize("captured", [False, True])
def test_draft_verify_accept(captured):
    import torch
    import paged_kv_cache_349_b200 as pa
    rng = np.random.default_rng(17)
    torch.manual_seed(17)
    B, Hq, Hkv, d, bs, n, steps = 3, 4, 2, 64, 8, 12, 5
    G, T = Hq // Hkv, B * n
    nb, mb, most = 64, 16, 5
    turns, gain = pa.pa_rope_frequencies(32, 10000.0)
    dturns = turns.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    k_cache, v_cache = (torch.full((nb, Hkv, bs, d), float("nan"), **bf) for _ in range(2))
    tables = torch.full((B, mb), -1, **i32)
    lens, cursor, free = torch.zeros(B, **i32), torch.zeros(1, **i32), i32_dev(rng.permutation(nb))
    flag = torch.zeros(1, **i32)

    # prompts: tables from the lengths, rotary positions and the cache write in one call
    prompt = np.array([5, 16, 23])
    P = int(prompt.sum())
    slots, pos, cu = torch.empty(P, **i32), torch.empty(P, **i32), torch.empty(B + 1, **i32)
    pa.pa_extend_tables(tables, lens, i32_dev(prompt), free, cursor, num_blocks=nb, block_size=bs, slot_mapping=slots,
                        positions=pos, cu_tokens=cu, err_flag=flag)
    qkv = torch.randn(P, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    q_rot = torch.empty(P, Hq, d, **bf)
    pa.pa_rope_and_cache(q, q_rot, k, v, k_cache, v_cache, slots, pos, dturns, gain=gain, err_flag=flag)
    k_rot = torch.empty(P, Hkv, d, **bf)
    pa.pa_rope(None, None, k, k_rot, pos, dturns, gain=gain)
    rows = [[], [], []]  # accepted (key, value) rows of each sequence, as cached
    at = 0
    for b in range(B):
        for i in range(prompt[b]):
            rows[b].append((k_rot[at].double().cpu().numpy(), v[at].double().cpu().numpy()))
            assert int(pos[at]) == i
            at += 1

    # the step's own buffers
    parents, cu_nodes = torch.empty(T, **i32), i32_dev(np.arange(B + 1) * n)
    masks, positions = torch.empty(T, 1, **i32), torch.empty(T, **i32)
    qkv = torch.empty(T, Hq + 2 * Hkv, d, **bf)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = torch.empty(T, Hq, d, **bf)
    add, path, tslots = torch.zeros(B, **i32), torch.zeros(B, most, **i32), torch.empty(T, **i32)
    scale = d ** -0.5
    cap = 128
    size = pa.pa_decode_tree_workspace_size(B, T, Hq, Hkv, d, bs, cap, n, 128)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")

    def verify():
        pa.pa_tree_masks(masks, positions, parents, cu_nodes, lens, max_nodes=n, err_flag=flag)
        pa.pa_rope(q, q, k, k, positions, dturns, gain=gain)
        pa.pa_decode_tree(out, q, k, v, k_cache, v_cache, tables, lens, cu_nodes, masks, max_seq_len=cap, max_nodes=n,
                          scale=scale, partition_tokens=128, workspace=ws, err_flag=flag)

    def accept():
        pa.pa_extend_tables(tables, lens, add, free, cursor, num_blocks=nb, block_size=bs, slot_mapping=tslots,
                            cu_tokens=cu, cu_rows=cu_nodes, path=path, err_flag=flag)
        pa.pa_reshape_and_cache(k.contiguous(), v.contiguous(), k_cache, v_cache, tslots, err_flag=flag)

    calls = [verify, accept]
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        parents.fill_(-1)
        qkv.zero_()
        with torch.cuda.stream(side):
            verify()
            accept()  # add is all zero: nothing changes
        torch.cuda.current_stream().wait_stream(side)
        graphs = []
        for call in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
            graphs.append(g)
        calls = [g.replay for g in graphs]

    for step in range(steps):
        tree = np.array([[max(-1, i - 1 - int(rng.integers(0, 3))) for i in range(n)] for _ in range(B)])
        parents.copy_(i32_dev(tree.reshape(-1)))
        qkv.copy_(torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16))
        calls[0]()
        got = out.double().cpu().numpy()
        qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
        for b in range(B):
            for i in range(n):
                chain, j = [], i
                while j >= 0:
                    chain.insert(0, j)
                    j = tree[b, j]
                assert int(positions[b * n + i]) == len(rows[b]) + len(chain) - 1
                ks = np.stack([r[0] for r in rows[b]] + [kh[b * n + j] for j in chain])
                vs = np.stack([r[1] for r in rows[b]] + [vh[b * n + j] for j in chain])
                for g in range(Hq):
                    o, A, e = attend(qh[b * n + i, g], ks[:, g // G], vs[:, g // G], scale)
                    tol = np.abs(o) * 2.0 ** -8 + A * (2.0 ** -8 + 4 * e + 2.0 ** -19)
                    assert (np.abs(got[b * n + i, g] - o) <= tol).all(), (step, b, i, g)
        # keep a path from the root of one node, of any length, none at all among them
        kept = []
        for b in range(B):
            i = int(rng.integers(0, n))
            chain = []
            while i >= 0:
                chain.insert(0, i)
                i = tree[b, i]
            kept.append(chain[:int(rng.integers(0, most + 1))])
            rows[b] += [(kh[b * n + j], vh[b * n + j]) for j in kept[-1]]
        add.copy_(i32_dev([len(c) for c in kept]))
        path.copy_(i32_dev([c + [-1] * (most - len(c)) for c in kept]))
        calls[1]()
        assert lens.tolist() == [len(r) for r in rows]
    assert int(flag.item()) == 0

    # the cache that the steps built, read by the ordinary decode
    q1 = torch.randn(B, Hq, d, device="cuda").to(torch.bfloat16)
    out1 = torch.empty(B, Hq, d, device="cuda")
    pa.pa_decode(out1, q1, k_cache, v_cache, tables, lens, max_seq_len=cap, scale=scale, partition_tokens=-1, err_flag=flag)
    got = out1.double().cpu().numpy()
    for b in range(B):
        for g in range(Hq):
            ks, vs = (np.stack([r[x] for r in rows[b]])[:, g // G] for x in (0, 1))
            o, A, e = attend(q1[b, g].double().cpu().numpy(), ks, vs, scale)
            assert (np.abs(got[b, g] - o) <= A * (2.0 ** -14 + 4 * e)).all()
    assert int(flag.item()) == 0
