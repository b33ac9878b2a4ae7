"""Rotary positions (pa_rope, pa_rope_and_cache[_fp8]) against the rotation in 64 bits.

Tolerances.  A rotated value is a c - b s of exact bf16 a, b.  cos and sin carry
the angle's fp32 rounding (2^-24 of a half turn: pi * 2^-24 < 2^-22) and their own
error (< 2^-22); the two products and the sum round to fp32.  Together below 2^-20 of
gain * (|a| + |b|).  Then one rounding: bf16 2^-8 of the value, E4M3 2^-4 of it, or half a
subnormal step (2^-10 codes).  Values that pass through, and v, keep their bits.
"""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import i32_dev

pytestmark = pytest.mark.gpu
ARITH = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def rotated(x, positions, turns, rotary, interleaved, gain):
    """x float64 [T, H, d] -> (rotated, the arithmetic's error bound)."""
    a = 2 * np.pi * positions.astype(np.float64)[:, None, None] * turns
    c, s = np.cos(a) * gain, np.sin(a) * gain
    lo, hi = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2),
                                                                              slice(rotary // 2, rotary))
    y, tol = x.copy(), np.zeros_like(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    tol[..., lo] = tol[..., hi] = ARITH * gain * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
    return y, tol


def close_bf16(got, want, tol):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8)).all(), err.max()


def inputs(T, Hq, Hkv, d, seed, fused=True):
    import torch
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    return parts if fused else tuple(p.contiguous() for p in parts)


def slots_for(T, nb, bs, seed):
    rng = np.random.default_rng(seed)
    s = rng.permutation(nb * bs)[:T].astype(np.int32)
    s[rng.random(T) < 0.1] = -1
    return s


@pytest.mark.parametrize("d,rotary", [(64, 16), (64, 64), (128, 32), (128, 96), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,bs", [(1, 4, 2, 16), (7, 40, 40, 8), (131, 8, 1, 64), (1203, 32, 8, 32)])
def test_rope_and_cache(d, rotary, interleaved, T, Hq, Hkv, bs):
    import torch
    import paged_kv_cache_349_b200 as pa
    q, k, v = inputs(T, Hq, Hkv, d, T + d + rotary)
    turns, gain = pa.pa_rope_frequencies(rotary, 10000.0, "by_parts", 4.0, 4096.0)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 1 << 20, size=T)
    nb = -(-T // bs) + 2
    slots = slots_for(T, nb, bs, T)
    kc = torch.full((nb, Hkv, bs, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    out = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = pa.launch_count()
    pa.pa_rope_and_cache(q, out, k, v, kc, vc, i32_dev(slots), i32_dev(pos), turns.cuda(), interleaved=interleaved,
                         gain=gain, err_flag=flag)
    assert pa.launch_count() - before == 1
    assert int(flag.item()) == 0
    tn = turns.numpy()
    want, tol = rotated(q.double().cpu().numpy(), pos, tn, rotary, interleaved, gain)
    close_bf16(out, want, tol)
    assert torch.equal(out[..., rotary:].view(torch.int16), q[..., rotary:].contiguous().view(torch.int16))
    want, tol = rotated(k.double().cpu().numpy(), pos, tn, rotary, interleaved, gain)
    kept = np.nonzero(slots >= 0)[0]
    rows = torch.from_numpy(slots[kept].astype(np.int64)).cuda()
    close_bf16(kc[rows // bs, :, rows % bs], want[kept], tol[kept])
    assert torch.equal(vc[rows // bs, :, rows % bs], v[torch.from_numpy(kept).cuda()])
    # every other pool row is as it was
    kc[rows // bs, :, rows % bs] = float("nan")
    vc[rows // bs, :, rows % bs] = float("nan")
    assert bool(kc.isnan().all()) and bool(vc.isnan().all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary,T,Hq,Hkv,bs", [(128, 128, 257, 32, 8, 16), (64, 32, 5, 4, 2, 8), (128, 48, 66, 0, 3, 32)])
def test_rope_and_cache_fp8(interleaved, d, rotary, T, Hq, Hkv, bs):
    import torch
    import paged_kv_cache_349_b200 as pa
    q, k, v = inputs(T, Hq, Hkv, d, T)
    turns, gain = pa.pa_rope_frequencies(rotary, 500000.0, "linear", 8.0)
    pos = np.random.default_rng(T).integers(0, 200000, size=T)
    nb = -(-T // bs) + 2
    slots = slots_for(T, nb, bs, T)
    kc = torch.full((nb, Hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    k_scale, v_scale = 0.004, 0.011  # k saturates in places
    out = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda") if Hq else None
    pa.pa_rope_and_cache_fp8(q if Hq else None, out, k, v, kc, vc, i32_dev(slots), i32_dev(pos), turns.cuda(),
                             interleaved=interleaved, gain=gain, k_scale=k_scale, v_scale=v_scale)
    tn = turns.numpy()
    if Hq:
        close_bf16(out, *rotated(q.double().cpu().numpy(), pos, tn, rotary, interleaved, gain))
    kept = np.nonzero(slots >= 0)[0]
    rows = torch.from_numpy(slots[kept].astype(np.int64)).cuda()
    want, tol = rotated(k.double().cpu().numpy(), pos, tn, rotary, interleaved, gain)
    got = kc[rows // bs, :, rows % bs].view(torch.float8_e4m3fn).double().cpu().numpy()
    w, t = want[kept] / np.float32(k_scale), tol[kept] / np.float32(k_scale)
    clipped = np.clip(w, -448.0, 448.0)
    # the code's own rounding, the reciprocal scale in fp32 (2^-22 of the value) and the rotation's error
    assert (np.abs(got - clipped) <= np.maximum(np.abs(clipped) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10)
            + np.abs(w) * 2.0 ** -22 + t * 1.1).all()
    bits = v[torch.from_numpy(kept).cuda()].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    codes = vc[rows // bs, :, rows % bs].cpu().numpy()
    assert np.array_equal(codes, oracle.quantize_e4m3(bits, v_scale))
    kc[rows // bs, :, rows % bs] = 0x7F
    vc[rows // bs, :, rows % bs] = 0x7F
    assert bool((kc == 0x7F).all()) and bool((vc == 0x7F).all())


@pytest.mark.parametrize("T", [1, 3, 64, 1000])
@pytest.mark.parametrize("fused", [False, True])
def test_rope_out_of_place_and_in_place(T, fused):
    import torch
    import paged_kv_cache_349_b200 as pa
    Hq, Hkv, d, rotary = 6, 3, 128, 64
    q, k, v = inputs(T, Hq, Hkv, d, T, fused)
    v0 = v.clone()
    turns, gain = pa.pa_rope_frequencies(rotary, 10000.0)
    pos = np.arange(T) + 31
    qo, ko = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hkv, d, dtype=torch.bfloat16,
                                                                                     device="cuda")
    tn = turns.numpy()
    args = (i32_dev(pos), turns.cuda())
    wq = rotated(q.double().cpu().numpy(), pos, tn, rotary, False, gain)
    wk = rotated(k.double().cpu().numpy(), pos, tn, rotary, False, gain)
    pa.pa_rope(q, qo, k, ko, *args, gain=gain)
    close_bf16(qo, *wq)
    close_bf16(ko, *wk)
    only = torch.empty_like(ko)
    pa.pa_rope(None, None, k, only, *args, gain=gain)
    assert torch.equal(only, ko)
    pa.pa_rope(q, q, k, k, *args, gain=gain)  # in place, also inside the projection's output
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, v0)


def test_far_and_extreme_positions():
    """Positions up to 2^31 - 1 and negative ones: the angle keeps its phase (fp64: 2^-53 * 2^28 turns = 2^-25)."""
    import torch
    import paged_kv_cache_349_b200 as pa
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=np.int64)
    T, d = len(pos), 128
    q, k, _ = inputs(T, 4, 2, d, 1)
    turns, gain = pa.pa_rope_frequencies(d, 10000.0)
    qo, ko = torch.empty(T, 4, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 2, d, dtype=torch.bfloat16,
                                                                                    device="cuda")
    pa.pa_rope(q, qo, k, ko, i32_dev(pos), turns.cuda(), gain=gain)
    # reduce the turns exactly before numpy's cosine: position * turns in extended precision
    frac = (pos.astype(np.longdouble)[:, None] * turns.numpy().astype(np.longdouble)) % 1.0
    a = 2 * np.pi * frac.astype(np.float64)[:, None]
    x = q.double().cpu().numpy()
    want = np.concatenate([x[..., :64] * np.cos(a) - x[..., 64:] * np.sin(a),
                           x[..., 64:] * np.cos(a) + x[..., :64] * np.sin(a)], -1)
    tol = np.tile(ARITH * (np.abs(x[..., :64]) + np.abs(x[..., 64:])), (1, 1, 2))
    close_bf16(qo, want, tol)
    assert torch.equal(qo[0], q[0]) and torch.equal(ko[0], k[0])  # position 0 turns nothing


def test_bad_slots_are_flagged_and_skipped():
    import torch
    import paged_kv_cache_349_b200 as pa
    q, k, v = inputs(4, 4, 2, 64, 9)
    turns, _ = pa.pa_rope_frequencies(64)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc, flag = kc.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(q, qo, k, v, kc, vc, i32_dev([32, -2, -1, 5]), i32_dev([0] * 4), turns.cuda(), err_flag=flag)
    assert int(flag.item()) == pa.PA_FLAG_BAD_SLOT
    assert torch.equal(qo, q)  # q is rotated whatever its slot is
    assert torch.equal(kc[0, :, 5], k[3]) and torch.equal(vc[0, :, 5], v[3])
    kc[0, :, 5] = 0
    assert not bool(kc.any())


def test_python_refusals():
    import torch
    import paged_kv_cache_349_b200 as pa
    q, k, v = inputs(4, 4, 2, 64, 9)
    turns = pa.pa_rope_frequencies(64)[0].cuda()
    pos, out = i32_dev([0] * 4), torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: pa.pa_rope(q, None, k, ko, pos, turns), lambda: pa.pa_rope(None, None, None, None, pos, turns),
                lambda: pa.pa_rope(q, out[:3], k, ko, pos, turns), lambda: pa.pa_rope(q, out, k, ko, pos[:2], turns),
                lambda: pa.pa_rope(q.transpose(0, 1), out.transpose(0, 1), None, None, pos, turns)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pa.pa_rope(q.float(), out, k, ko, pos, turns), lambda: pa.pa_rope(q.cpu(), out, k, ko, pos, turns),
                lambda: pa.pa_rope(q, out, k, ko, pos.long(), turns), lambda: pa.pa_rope(q, out, k, ko, pos, turns.float())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(pa.PaError):
        pa.pa_rope(q, out, k, ko, pos, turns[:5])  # 10 values: not a multiple of 16
