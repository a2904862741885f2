"""Language-model entry points (prompt_attention, key_weights,
prefix_attention, evict) against their definitions in 64 bits.

Tolerances, per output value, from the arithmetic the header promises: with u
half a step of the 16-bit type (2^-8 bf16, 2^-11 fp16),
  logit     fp32 sum of d products in any order: |dx| <= d 2^-23 c sum|q_e k_e|
  weight    exp of it and of the normaliser: relative 2 |dx| + 2^-19
  O         each weight rounded to the type (u) and O once (u):
            u |O| + (u + 2 |dx| + 2^-19) sum_j p_j |v_j|, and for fp16, whose
            smallest step is 2^-24, 2^-25 sum_j |v_j| more
  lse       |dx| + 2^-22 |lse| + 2^-20
  key weight  sum over its N rows of p (|dx| + 2^-21 |lse| + 2^-19), and N 2^-24
            of the sum for adding it up in fp32
"""
import math
import os
import threading

import numpy as np
import pytest
import torch

import block_sparse_attention_head_b200 as ig

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HALF_STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_attention_head_b200 import build
    build.build()
    ig.lib()
    yield
    ig.device_status()


def normal(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def cu(lens, start=0):
    return torch.tensor(np.cumsum([start] + list(lens)), dtype=torch.int32, device="cuda")


def attend(q, k, v, scale, seen=None):
    """One head in 64 bits: O, lse, weights, and the tolerances of O and lse."""
    u, fp16 = HALF_STEP[q.dtype], q.dtype == FP
    q, k, v = q.double(), k.double(), v.double()
    x = q @ k.t() * scale
    dx = q.shape[1] * 2.0 ** -23 * scale * (q.abs() @ k.abs().t())
    if seen is not None:
        x = x.masked_fill(~seen, -math.inf)
        dx = dx * seen
    dx = dx.amax(1, keepdim=True) if k.shape[0] else torch.zeros(q.shape[0], 1, dtype=q.dtype, device=q.device)
    lse = torch.logsumexp(x, 1, keepdim=True)
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    o = p @ v
    tol = u * o.abs() + (u + 2 * dx + 2.0 ** -19) * (p @ v.abs())
    if fp16:
        tol = tol + 2.0 ** -25 * v.abs().sum(0)
    lse, dx = lse[:, 0], dx[:, 0]
    tol_lse = dx + 2.0 ** -22 * torch.where(lse == -math.inf, torch.zeros_like(lse), lse).abs() + 2.0 ** -20
    return o, lse, p, tol, tol_lse, dx


def within(got, want, tol, what):
    got, want, tol = got.double(), want.double(), tol.double() + 1e-30
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    bad = ~((got - want).abs() <= tol) & ~inf
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {((got - want).abs() / tol)[~inf].max():.2f}x"


def causal_mask(nq, nk):
    return torch.arange(nk, device="cuda")[None] <= torch.arange(nq, device="cuda")[:, None] + nk - nq


def check_prompt(q, k, v, qs, ks, causal, O, lse, scale=None, q0=0, k0=0, weights=None, before=None):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    G = q.shape[1] // k.shape[1]
    W = None if weights is None else before.double().clone()
    Wtol = None if weights is None else 2.0 ** -22 * before.double().abs()
    i, j = q0, k0
    for nq, nk in zip(qs, ks):
        seen = causal_mask(nq, nk) if causal else None
        for h in range(q.shape[1]):
            o, l, p, tol, tol_l, dx = attend(q[i:i + nq, h], k[j:j + nk, h // G], v[j:j + nk, h // G], scale, seen)
            if O is not None:
                within(O[i:i + nq, h], o, tol, f"O of head {h}, rows {i}:{i + nq}")
                within(lse[h, i:i + nq], l, tol_l, f"lse of head {h}")
            if W is not None:
                l = torch.where(l == -math.inf, torch.zeros_like(l), l)
                W[h // G, j:j + nk] += p.sum(0)
                Wtol[h // G, j:j + nk] += (p * (dx + 2.0 ** -21 * l.abs() + 2.0 ** -19 + tol_l)[:, None]).sum(0)
                Wtol[h // G, j:j + nk] += G * nq * 2.0 ** -24 * p.sum(0)
        i, j = i + nq, j + nk
    if W is not None:
        within(weights, W, Wtol, "weights")


PROMPTS = {
    # name: (query lengths, key lengths, Hq, Hkv, d)
    "one_token": ([1], [1], 1, 1, 64),
    "one_query": ([1], [700], 8, 2, 128),
    "empty_sequences": ([1, 0, 5, 0], [1, 3, 5, 0], 4, 4, 64),
    "no_keys": ([7, 130], [0, 130], 4, 2, 128),
    "fewer_keys_than_queries": ([200, 3], [50, 1], 2, 1, 64),
    "exact_tiles": ([128, 256], [128, 256], 2, 2, 128),
    "one_past_tiles": ([129, 257, 1], [129, 257, 129], 3, 1, 128),
    "odd_groups": ([61, 300], [61, 300], 10, 2, 64),
    "wide_group": ([5, 33], [40, 33], 71, 1, 128),
    "chunk": ([40, 257], [900, 1300], 6, 2, 128),
    "many_short": ([1 + (7 * i) % 23 for i in range(70)], [1 + (7 * i) % 23 + i for i in range(70)], 8, 2, 64),
    "steps": ([1] * 33, [1 + 37 * i for i in range(33)], 16, 2, 128),
    "long": ([1500], [4100], 4, 2, 128),
    "long_few_rows": ([3], [9001], 5, 1, 64),
    "ragged_last": ([257, 300], [2100, 2200], 50, 50, 64),
}


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompt_attention_and_key_weights(name, causal, dtype):
    qs, ks, Hq, Hkv, d = PROMPTS[name]
    q, k, v = (normal(i, n, H, d, dtype=dtype, scale=s) for i, n, H, s in
               ((1, sum(qs), Hq, 1.2), (2, sum(ks), Hkv, 1.2), (3, sum(ks), Hkv, 1.0)))
    O, lse = ig.prompt_attention(q, k, v, cu(qs), cu(ks), causal=causal)
    check_prompt(q, k, v, qs, ks, causal, O, lse)
    before = normal(4, Hkv, sum(ks), dtype=torch.float32).abs()
    w = ig.key_weights(q, k, lse, cu(qs), cu(ks), before.clone(), causal=causal)
    check_prompt(q, k, v, qs, ks, causal, None, None, weights=w, before=before)
    ig.device_status()


def test_prompt_scale_and_spread_logits():
    # logits over +-60: the running maximum moves by large steps, small weights vanish
    qs = ks = [333]
    q, k, v = normal(1, 333, 4, 64, scale=2.0), normal(2, 333, 2, 64, scale=2.0), normal(3, 333, 2, 64)
    k[::50] *= 3
    O, lse = ig.prompt_attention(q, k, v, cu(qs), cu(ks), softmax_scale=0.4)
    check_prompt(q, k, v, qs, ks, True, O, lse, scale=0.4)
    w = ig.key_weights(q, k, lse, cu(qs), cu(ks), torch.zeros(2, 333, device="cuda"), softmax_scale=0.4)
    check_prompt(q, k, v, qs, ks, True, None, None, scale=0.4, weights=w, before=torch.zeros_like(w))


@pytest.mark.parametrize("layout", ["fused", "head_major", "padded_rows"])
def test_prompt_strided_views(layout):
    qs, ks, Hq, Hkv, d = [100, 77], [100, 77], 6, 2, 64
    T = sum(qs)
    if layout == "fused":  # one projection's output
        x = normal(1, T, (Hq + 2 * Hkv) * d)
        q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([Hq * d, Hkv * d, Hkv * d], 1))
        out = torch.zeros(T, Hq + 1, d, dtype=BF, device="cuda")[:, 1:]
    elif layout == "head_major":
        q, k, v = (normal(i, H, T, d).transpose(0, 1) for i, H in ((1, Hq), (2, Hkv), (3, Hkv)))
        out = torch.zeros(Hq, T, d, dtype=BF, device="cuda").transpose(0, 1)
    else:
        q, k, v = (normal(i, T, H, d + 8)[..., :d] for i, H in ((1, Hq), (2, Hkv), (3, Hkv)))
        out = torch.zeros(T, Hq, d + 40, dtype=BF, device="cuda")[..., :d]
    O, lse = ig.prompt_attention(q, k, v, cu(qs), cu(ks), out=out)
    assert O.data_ptr() == out.data_ptr()
    check_prompt(q, k, v, qs, ks, True, O, lse)
    w = ig.key_weights(q, k, lse, cu(qs), cu(ks), torch.zeros(Hkv, T, device="cuda"))
    check_prompt(q, k, v, qs, ks, True, None, None, weights=w, before=torch.zeros_like(w))
    ref, _ = ig.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu(qs), cu(ks))
    assert torch.equal(ref, O)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_of_no_sequence_are_left_and_never_read_into_results(causal):
    """Rows before, between tiles of, and behind the sequences hold NaN and
    infinities; outputs there keep what they had."""
    qs, ks, Hq, Hkv, d = [70, 30], [70, 130], 4, 2, 128
    Tq, Tk, q0, k0 = 150, 260, 11, 9
    q, k, v = normal(1, Tq, Hq, d), normal(2, Tk, Hkv, d), normal(3, Tk, Hkv, d)
    for t, lo, n in ((q, q0, sum(qs)), (k, k0, sum(ks)), (v, k0, sum(ks))):
        t[:lo] = math.nan
        t[lo + n:] = math.inf
    out = torch.full((Tq, Hq, d), 7.0, dtype=BF, device="cuda")
    lse = torch.full((Hq, Tq), 7.0, device="cuda")
    ig.prompt_attention(q, k, v, cu(qs, q0), cu(ks, k0), causal=causal, out=out, lse=lse)
    check_prompt(q, k, v, qs, ks, causal, out, lse, q0=q0, k0=k0)
    w = torch.full((Hkv, Tk), 2.0, device="cuda")
    ig.key_weights(q, k, lse, cu(qs, q0), cu(ks, k0), w, causal=causal)
    check_prompt(q, k, v, qs, ks, causal, None, None, q0=q0, k0=k0, weights=w, before=torch.full_like(w, 2.0))
    for rows in (slice(0, q0), slice(q0 + sum(qs), None)):
        assert (out[rows] == 7).all() and (lse[:, rows] == 7).all()
    assert (w[:, :k0] == 2).all() and (w[:, k0 + sum(ks):] == 2).all()
    # a neighbour's NaN stays with the neighbour
    k[k0 + 70:k0 + 200] = math.nan
    v[k0 + 70:k0 + 200] = math.nan
    O2, lse2 = ig.prompt_attention(q, k, v, cu(qs, q0), cu(ks, k0), causal=causal)
    assert torch.equal(O2[q0:q0 + 70], out[q0:q0 + 70]) and torch.equal(lse2[:, q0:q0 + 70], lse[:, q0:q0 + 70])


def test_prompt_no_queries_or_no_keys_at_all():
    q, k = normal(1, 0, 4, 64), normal(2, 5, 2, 64)
    O, lse = ig.prompt_attention(q, k, k, cu([0]), cu([5]))
    assert O.shape == (0, 4, 64) and lse.shape == (4, 0)
    q, k = normal(1, 5, 4, 64), normal(2, 0, 2, 64)
    O, lse = ig.prompt_attention(q, k, k, cu([5]), cu([0]))
    assert (O == 0).all() and (lse == -math.inf).all()
    ig.key_weights(q, k, lse, cu([5]), cu([0]), torch.zeros(2, 0, device="cuda"))
    ig.device_status()


@pytest.mark.parametrize("d", [64, 128])
def test_split_keys_without_any_sequence_then_a_call_with_new_ends(d):
    """No row and no key in a sequence where the keys are split over CTAs:
    nothing is written, and the ends and the workspace may change right behind."""
    Tq, Tk, Hq, Hkv = 700, 9000, 4, 2
    q, k, v = normal(1, Tq, Hq, d), normal(2, Tk, Hkv, d), normal(3, Tk, Hkv, d)
    ends_q, ends_k = cu([Tq]), cu([Tk])
    want, want_lse = ig.prompt_attention(q, k, v, ends_q, ends_k)
    want_w = ig.key_weights(q, k, want_lse, ends_q, ends_k, torch.zeros(Hkv, Tk, device="cuda"))
    work = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    cu_q, cu_k = cu([0]), cu([0])
    out = torch.full((Tq, Hq, d), 7.0, dtype=BF, device="cuda")
    lse = torch.full((Hq, Tq), 7.0, device="cuda")
    w = torch.full((Hkv, Tk), 2.0, device="cuda")
    for _ in range(20):
        ig.prompt_attention(q, k, v, cu_q, cu_k, out=out, lse=lse, workspace=work)
        cu_q.copy_(ends_q), cu_k.copy_(ends_k), work.fill_(255)
        cu_q.zero_(), cu_k.zero_()
        ig.key_weights(q, k, lse, cu_q, cu_k, w, workspace=work)
        cu_q.copy_(ends_q), cu_k.copy_(ends_k), work.fill_(255)
        cu_q.zero_(), cu_k.zero_()
    assert (out == 7).all() and (lse == 7).all() and (w == 2).all()
    cu_q.copy_(ends_q), cu_k.copy_(ends_k)
    ig.prompt_attention(q, k, v, cu_q, cu_k, out=out, lse=lse, workspace=work)
    ig.key_weights(q, k, lse, cu_q, cu_k, w.zero_(), workspace=work)
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(w, want_w)
    ig.device_status()


def test_prompt_bad_ends_are_reported_and_stay_in_range():
    q, k = normal(1, 20, 2, 64), normal(2, 20, 2, 64)
    bad = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    ig.prompt_attention(q, k, k, bad, bad)
    with pytest.raises(ig.InstaGenError, match="device check"):
        ig.device_status()
    ig.device_status()


# -------------------------------------------------------------------- steps
STEPS = {
    # name: (B, P, lens, cap, Hq, Hkv, d)
    "one": (1, 0, [1], 1, 1, 1, 64),
    "nothing": (2, 0, [0, 0], 4, 4, 2, 64),
    "no_cache": (3, 70, [0, 0, 0], 0, 4, 2, 128),
    "one_alone": (1, 0, [300], 512, 8, 2, 64),
    "some_empty": (5, 0, [0, 1, 64, 65, 127], 128, 8, 2, 128),
    "tiles": (4, 128, [128, 256, 129, 1], 256, 8, 8, 128),
    "prefix_only_some": (3, 1000, [0, 5, 0], 8, 6, 2, 128),
    "odd": (7, 333, [3 * i for i in range(7)], 19, 15, 3, 64),
    "wide_group": (3, 50, [40, 41, 300], 301, 71, 1, 128),
    "ungrouped": (9, 200, [17 * i for i in range(9)], 140, 12, 12, 128),
    "big_batch": (130, 700, [(29 * i) % 90 for i in range(130)], 90, 8, 2, 128),
    "long_prefix": (40, 9000, [50 + i for i in range(40)], 100, 8, 2, 64),
    "long_own": (2, 0, [20000, 5001], 20003, 8, 2, 128),
    "long_both": (20, 5000, [3000 - 100 * i for i in range(20)], 3001, 4, 1, 128),
    "tall_prefix": (70, 4111, [(11 * i) % 33 for i in range(70)], 33, 20, 4, 128),
    "crowded": (130, 3001, [(7 * i) % 21 for i in range(130)], 21, 16, 8, 64),
    "many_long": (150, 3, [5001 - 33 * i for i in range(150)], 5001, 4, 2, 64),
}


def step_inputs(name, dtype):
    B, P, lens, cap, Hq, Hkv, d = STEPS[name]
    q = normal(1, B, Hq, d, dtype=dtype, scale=1.2)
    kp, vp = normal(2, Hkv, P, d, dtype=dtype, scale=1.2), normal(3, Hkv, P, d, dtype=dtype)
    kc, vc = normal(4, B, Hkv, cap, d, dtype=dtype, scale=1.2), normal(5, B, Hkv, cap, d, dtype=dtype)
    for b, n in enumerate(lens):  # what is behind the length never matters
        kc[b, :, n:], vc[b, :, n:] = math.nan, math.inf
    return q, kp, vp, kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_step(q, kp, vp, kc, vc, lens, O, lse, before=None, weights=None):
    B, Hq, d = q.shape
    Hkv, P = kc.shape[1], 0 if kp is None else kp.shape[1]
    G = Hq // Hkv
    W = None if weights is None else before.double().clone()
    Wtol = None if weights is None else 2.0 ** -22 * before.double().abs()
    for b, n in enumerate(lens.tolist()):
        for hk in range(Hkv):
            k, v = kc[b, hk, :n], vc[b, hk, :n]
            if P:
                k, v = torch.cat([kp[hk], k]), torch.cat([vp[hk], v])
            hs = slice(hk * G, hk * G + G)
            o, l, p, tol, tol_l, dx = attend(q[b, hs], k, v, 1 / math.sqrt(d))
            within(O[b, hs], o, tol, f"O of sequence {b}, heads {hs}")
            within(lse[b, hs], l, tol_l, f"lse of sequence {b}")
            if W is not None:
                W[b, hk, :n] += p[:, P:].sum(0)
                l = torch.where(l == -math.inf, torch.zeros_like(l), l)
                Wtol[b, hk, :n] += (p[:, P:] * (dx + 2.0 ** -21 * l.abs() + 2.0 ** -19 + tol_l)[:, None]).sum(0) \
                    + G * 2.0 ** -24 * p[:, P:].sum(0)
    if W is not None:
        within(weights, W, Wtol, "weights")


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("keep", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("name", list(STEPS))
def test_prefix_attention(name, keep, dtype):
    args = step_inputs(name, dtype)
    B, Hkv, cap = args[3].shape[:3]
    before = normal(6, B, Hkv, cap, dtype=torch.float32).abs()
    w = before.clone() if keep else None
    O, lse = ig.prefix_attention(*args, weights=w)
    check_step(*args, O, lse, before, w)
    ig.device_status()


def test_prefix_attention_views_and_no_prefix():
    q, kp, vp, kc, vc, lens = step_inputs("odd", BF)
    B, Hq, d = q.shape
    O, lse = ig.prefix_attention(q, kp, vp, kc, vc, lens)
    # q out of a fused projection, the prefix out of a longer cache
    fused = torch.zeros(B, (Hq + 6) * d, dtype=BF, device="cuda")
    fused[:, :Hq * d] = q.flatten(1)
    long_k, long_v = (torch.full((t.shape[0], 400, d), math.nan, dtype=BF, device="cuda") for t in (kp, vp))
    long_k[:, :kp.shape[1]], long_v[:, :kp.shape[1]] = kp, vp
    O2, lse2 = ig.prefix_attention(fused[:, :Hq * d].unflatten(1, (Hq, d)), long_k[:, :kp.shape[1]],
                                   long_v[:, :kp.shape[1]], kc, vc, lens)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    O3, lse3 = ig.prefix_attention(q, None, None, kc, vc, lens)
    check_step(q, None, None, kc, vc, lens, O3, lse3)


def test_prefix_attention_offsets_past_32_bits():
    # the last head's rows start past 2^31 elements (2^32 bytes) into the cache
    B, Hkv, cap, d, n = 2, 8, 1100000, 128, 300
    kc, vc = (torch.empty(B, Hkv, cap, d, dtype=BF, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    kc[:, :, :n], vc[:, :, :n] = normal(1, B, Hkv, n, d), normal(2, B, Hkv, n, d)
    q, lens = normal(3, B, 8, d), torch.tensor([n, n - 7], dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, cap, device="cuda")
    O, lse = ig.prefix_attention(q, None, None, kc, vc, lens, weights=w)
    small = [t[:, :, :n].contiguous() for t in (kc, vc, w)]
    check_step(q, None, None, small[0], small[1], lens, O, lse, torch.zeros_like(small[2]), small[2])
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, Hkv, cap).contiguous()
    want = [t.clone() for t in (small[0], small[1], small[2], pos[:, :, :n].contiguous(), lens)]
    ig.evict(kc, vc, w, pos, lens, 250, 20)
    check_evict(want, [kc[:, :, :n], vc[:, :, :n], w[:, :, :n], pos[:, :, :n], lens], 250, 20)
    ig.device_status()


def test_prefix_attention_bad_lengths_are_reported_and_stay_in_range():
    q, kp, vp, kc, vc, lens = step_inputs("tiles", BF)
    ig.prefix_attention(q, kp, vp, kc, vc, lens + 1000)
    with pytest.raises(ig.InstaGenError, match="device check"):
        ig.device_status()


# ----------------------------------------------------------------- eviction
def evicted(before, budget, recent):
    """The definition, slot by slot, on the host (outputs start as copies of the inputs)."""
    k, v, w, pos, lens = before
    out = [k.clone(), v.clone(), w.clone(), pos.clone(), lens.clamp(max=budget)]
    wn, pn = w.cpu().numpy(), pos.cpu().numpy()
    for b, n in enumerate(lens.tolist()):
        if n <= budget:
            continue
        for h in range(k.shape[1]):
            x, t = wn[b, h, :n], pn[b, h, :n].astype(np.int64)
            order = sorted(range(n), key=lambda i: (not t[i] > t.max() - recent,
                                                    math.inf if math.isnan(x[i]) else -float(x[i]),
                                                    math.isnan(x[i]), i))
            kept = set(order[:budget])
            freed = [i for i in range(budget) if i not in kept]
            moved = [i for i in range(budget, n) if i in kept]
            assert len(freed) == len(moved)
            if freed:
                for x_in, x_out in zip(before[:4], out[:4]):
                    x_out[b, h, freed] = x_in[b, h, moved]
    return out


def check_evict(before, after, budget, recent):
    want = evicted(before, budget, recent)
    assert torch.equal(after[4], want[4])
    for b, n in enumerate(want[4].tolist()):
        for got, ref in zip(after[:4], want[:4]):
            assert torch.equal(torch.nan_to_num(got[b, :, :n].float()), torch.nan_to_num(ref[b, :, :n].float()))


def evict_inputs(B, Hkv, cap, d, lens, kind, dtype=BF):
    k, v = normal(1, B, Hkv, cap, d, dtype=dtype), normal(2, B, Hkv, cap, d, dtype=dtype)
    w = normal(3, B, Hkv, cap, dtype=torch.float32).abs()
    if kind == "ties":
        w = (w * 3).round()
    elif kind == "equal":
        w = torch.ones_like(w)
    elif kind == "odd":  # infinities, NaN, both zeros, negatives
        w = normal(3, B, Hkv, cap, dtype=torch.float32)
        w[..., ::7], w[..., 1::11], w[..., 2::13], w[..., 3::9], w[..., 4::17] = math.nan, math.inf, -math.inf, 0.0, -0.0
    g = torch.Generator(device="cuda").manual_seed(9)
    pos = torch.rand(B, Hkv, cap, generator=g, device="cuda").argsort(-1).to(torch.int32) - 50
    return [k, v, w, pos, torch.tensor(lens, dtype=torch.int32, device="cuda")]


EVICTS = {
    # name: (B, Hkv, cap, d, lens, budget, recent)
    "one_key": (1, 1, 1, 64, [1], 1, 0),
    "two_to_one": (1, 2, 2, 128, [2], 1, 0),
    "one_over": (3, 2, 101, 128, [101, 100, 7], 100, 10),
    "nothing_to_do": (2, 2, 64, 64, [64, 0], 64, 5),
    "all_recent": (1, 3, 200, 128, [200], 50, 50),
    "recent_beyond_budget": (2, 1, 300, 64, [300, 61], 60, 1000),
    "half": (2, 3, 1000, 128, [999, 731], 500, 100),
    "to_few": (4, 2, 5000, 128, [5000, 4097, 30, 1], 33, 8),
    "more_than_a_pass": (1, 2, 20011, 64, [20001], 9000, 64),
    "long": (1, 1, 70001, 64, [70000], 1024, 128),
}


@pytest.mark.parametrize("place", [True, False], ids=["in_place", "copy"])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("name", list(EVICTS))
def test_evict(name, kind, place):
    B, Hkv, cap, d, lens, budget, recent = EVICTS[name]
    t = evict_inputs(B, Hkv, cap, d, lens, kind)
    before = [x.clone() for x in t]
    if place:
        got = ig.evict(*t, budget, recent)
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, t))
    else:
        m = budget + 3
        out = (torch.full((B, Hkv, m, d), 9.0, dtype=BF, device="cuda"), torch.full((B, Hkv, m, d), 9.0, dtype=BF, device="cuda"),
               torch.full((B, Hkv, m), 9.0, device="cuda"), torch.full((B, Hkv, m), 9, dtype=torch.int32, device="cuda"),
               torch.full((B,), 9, dtype=torch.int32, device="cuda"))
        got = ig.evict(*t, budget, recent, out=out)
        for a, b in zip(t, before):  # inputs untouched
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
        for b, n in enumerate(got[4].tolist()):  # the rest of the output too
            assert all((x[b, :, n:] == 9).all() for x in got[:4])
    check_evict(before, got, budget, recent)
    ig.device_status()


# ----------------------------------------------------------------- together
def test_a_prompt_then_steps_with_a_full_cache():
    """Prompts -> key weights -> eviction into small caches -> steps behind a
    shared prefix that add weights -> eviction in place, each against the
    definition on the state before it."""
    Hq, Hkv, d, budget, cap = 8, 2, 64, 96, 100
    qs = [150, 90, 260]
    q, k, v = normal(1, sum(qs), Hq, d), normal(2, sum(qs), Hkv, d), normal(3, sum(qs), Hkv, d)
    O, lse = ig.prompt_attention(q, k, v, cu(qs), cu(qs))
    w = ig.key_weights(q, k, lse, cu(qs), cu(qs), torch.zeros(Hkv, sum(qs), device="cuda"))
    check_prompt(q, k, v, qs, qs, True, O, lse, weights=w, before=torch.zeros_like(w))
    most, B = max(qs), len(qs)
    big = [torch.zeros(B, Hkv, most, d, dtype=BF, device="cuda"), torch.zeros(B, Hkv, most, d, dtype=BF, device="cuda"),
           torch.zeros(B, Hkv, most, device="cuda"), torch.zeros(B, Hkv, most, dtype=torch.int32, device="cuda"),
           torch.tensor(qs, dtype=torch.int32, device="cuda")]
    at = 0
    for b, n in enumerate(qs):
        big[0][b, :, :n], big[1][b, :, :n] = k[at:at + n].transpose(0, 1), v[at:at + n].transpose(0, 1)
        big[2][b, :, :n], big[3][b, :, :n] = w[:, at:at + n], torch.arange(n, device="cuda")
        at += n
    cache = ig.evict(*big, budget, 16, out=tuple(
        torch.zeros(B, Hkv, cap, *t.shape[3:], dtype=t.dtype, device="cuda") for t in big[:4]) + (big[4].clone(),))
    check_evict(big, cache, budget, 16)
    kc, vc, wc, pos, lens = cache
    kp, vp = normal(7, Hkv, 500, d), normal(8, Hkv, 500, d)
    rows = torch.arange(B, device="cuda")
    for step in range(9):
        kc[rows, :, lens.long()], vc[rows, :, lens.long()] = normal(20 + step, B, Hkv, d), normal(40 + step, B, Hkv, d)
        wc[rows, :, lens.long()] = 0
        pos[rows, :, lens.long()] = (torch.tensor(qs, device="cuda")[:, None] + step).to(torch.int32).expand(B, Hkv)
        lens += 1
        before, x = wc.clone(), normal(60 + step, B, Hq, d)
        O, lse = ig.prefix_attention(x, kp, vp, kc, vc, lens, weights=wc)
        check_step(x, kp, vp, kc, vc, lens, O, lse, before, wc)
        if int(lens.max()) == cap:
            state = [t.clone() for t in (kc, vc, wc, pos, lens)]
            ig.evict(kc, vc, wc, pos, lens, budget, 16)
            check_evict(state, (kc, vc, wc, pos, lens), budget, 16)
    ig.device_status()


def _calls():
    """One call of every entry point on static buffers (workspaces included): (inputs to change, call, outputs)."""
    qs, ks = [150, 33, 1], [400, 33, 200]
    q, k, v = normal(1, sum(qs), 8, 64), normal(2, sum(ks), 2, 64), normal(3, sum(ks), 2, 64)
    cq, ck, w = cu(qs), cu(ks), torch.zeros(2, sum(ks), device="cuda")
    s = step_inputs("long_both", BF)
    sw = torch.zeros(s[3].shape[:3], device="cuda")
    e = evict_inputs(2, 3, 1000, 128, [999, 731], "ties")
    eo = tuple(torch.zeros(2, 3, 500, *t.shape[3:], dtype=t.dtype, device="cuda") for t in e[:4]) + (e[4].clone(),)

    def call():
        o, lse = ig.prompt_attention(q, k, v, cq, ck)
        ig.key_weights(q, k, lse, cq, ck, w.zero_())
        so, sl = ig.prefix_attention(*s, weights=sw.zero_())
        ig.evict(*e, 500, 50, out=eo)
        return (o, lse, w, so, sl, sw) + eo

    return (q, k, v, s[0], s[3], e[2]), call


def test_capture_and_replay_with_new_contents():
    inputs, call = _calls()
    want_old = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want_old))
    for t in inputs:
        t.copy_(t.flip(0))
    graph.replay()
    got = [t.clone() for t in outs]
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(got, want))
    ig.device_status()


def test_two_streams_at_once_and_again_the_same_bits():
    pairs = [_calls() for _ in range(2)]
    for t in pairs[1][0]:
        t.copy_(t.flip(0))
    want = [[t.clone() for t in call()] for _, call in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, (_, call) in zip(streams, pairs):
            with torch.cuda.stream(st):
                got.append([t.clone() for t in call()])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(g, w))
    ig.device_status()


def test_evict_from_four_threads_with_caches_of_different_size():
    """Host threads with a stream and a workspace each, whose calls ask for
    different amounts of shared memory (150 caches: no cluster)."""
    B, Hkv, d, times = 75, 2, 64, 2000
    L, stores, errors, start = ig.lib(), [], [], threading.Barrier(4)
    for cap in (12000, 20000, 30000, 40000):
        t = [torch.zeros(B, Hkv, cap, d, dtype=BF, device="cuda"), torch.zeros(B, Hkv, cap, d, dtype=BF, device="cuda"),
             torch.rand(B, Hkv, cap, device="cuda"),
             torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, Hkv, cap).contiguous(),
             torch.full((B,), 40, dtype=torch.int32, device="cuda")]
        t[0][:, :, :40], t[1][:, :, :40] = normal(1, B, Hkv, 40, d), normal(2, B, Hkv, 40, d)
        before = [x[:, :, :40].clone() if x.dim() > 1 else x.clone() for x in t]
        stores.append((t, before, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(t, _, ws, stream):  # (the C entry, so that the threads meet inside it and not at the interpreter's lock)
        p = bytes(ig.CacheParams(B, Hkv, Hkv, d, 0, t[0].shape[2], 0, 1.0, Hkv * d, 0))
        at = [x.data_ptr() for x in t]
        start.wait()
        for _ in range(times):
            rc = L.instagen_evict(*at, p, 30, 5, *at, t[0].shape[2], ws.data_ptr(), ws.numel(), stream.cuda_stream)
            if rc:
                errors.append((t[0].shape[2], rc))

    threads = [threading.Thread(target=work, args=s) for s in stores]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for t, before, _, _ in stores:  # (from the second call on there is nothing to evict)
        check_evict(before, [x[:, :, :40] if x.dim() > 1 else x for x in t], 30, 5)
    ig.device_status()


@pytest.mark.parametrize("Tk", [700, 4096, 100000])
def test_no_queries_before_many_keys(Tk):
    q, k = normal(1, 0, 8, 64), normal(2, Tk, 8, 64)
    O, lse = ig.prompt_attention(q, k, k, cu([0]), cu([Tk]))
    assert O.shape == (0, 8, 64) and lse.shape == (8, 0)
    w = ig.key_weights(q, k, lse, cu([0]), cu([Tk]), torch.full((8, Tk), 2.0, device="cuda"))
    assert (w == 2).all()
    ig.device_status()


# --------------------------------------------------- logits that are not finite
def nan_rows(got, bad, what):
    """Rows [..., rows] (or rows with a last dimension) that are NaN: exactly those of bad."""
    assert torch.equal(torch.isnan(got.float()), bad), what


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq", [100, 300])  # one row tile, two
def test_a_nan_key_shows_in_every_row_that_sees_it(nq, dtype):
    nk, Hq, Hkv, d = 640, 2, 1, 64
    q, k, v = normal(1, nq, Hq, d, dtype=dtype), normal(2, nk, Hkv, d, dtype=dtype), normal(3, nk, Hkv, d, dtype=dtype)
    for key in (0, 5, 6, 7, 134, 255, 262, 390):  # in tiles without a mask
        x = k.clone()
        x[key, 0, 3] = math.nan
        O, lse = ig.prompt_attention(q, x, v, cu([nq]), cu([nk]), causal=False)
        assert torch.isnan(O).all() and torch.isnan(lse).all(), key
        # causal with as many keys as queries: the rows before do not see it
        O, lse = ig.prompt_attention(q, x[:nq], v[:nq], cu([nq]), cu([nq]))
        want = torch.arange(nq, device="cuda") >= key
        nan_rows(lse, want.expand(Hq, nq), key)
        nan_rows(O, want[:, None, None].expand(nq, Hq, d), key)
    ig.device_status()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_a_nan_query_shows_in_the_weights_of_the_keys_it_sees(dtype):
    nq, nk, d = 300, 700, 64
    q, k = normal(1, nq, 1, d, dtype=dtype), normal(2, nk, 1, d, dtype=dtype)
    _, lse = ig.prompt_attention(q, k, k, cu([nq]), cu([nk]))
    for row in (0, 1, 2, 3, 130, 137, 299):
        x = q.clone()
        x[row, 0, 5] = math.nan
        w = ig.key_weights(x, k, lse, cu([nq]), cu([nk]), torch.zeros(1, nk, device="cuda"))
        nan_rows(w[0], torch.arange(nk, device="cuda") <= row + nk - nq, row)


def test_rows_without_lse_add_nothing_to_the_weights():
    """lse = -inf: rows that a caller leaves out, here in tiles without a mask."""
    nq, nk, Hq, Hkv, d = 300, 900, 4, 2, 128
    q, k = normal(1, nq, Hq, d), normal(2, nk, Hkv, d)
    _, lse = ig.prompt_attention(q, k, k, cu([nq]), cu([nk]))
    none = torch.full_like(lse, -math.inf)
    w = ig.key_weights(q, k, none, cu([nq]), cu([nk]), torch.zeros(Hkv, nk, device="cuda"))
    assert (w == 0).all()
    some = lse.clone()
    some[:, 50:] = -math.inf
    w = ig.key_weights(q, k, some, cu([nq]), cu([nk]), torch.zeros(Hkv, nk, device="cuda"), causal=False)
    want = ig.key_weights(q[:50], k, lse[:, :50].contiguous(), cu([50]), cu([nk]), torch.zeros(Hkv, nk, device="cuda"),
                          causal=False)
    within(w, want.double(), 200 * 2.0 ** -23 * want.double(), "weights")  # the same terms, added in another order


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq", [100, 300])
def test_logits_of_minus_infinity_weigh_nothing(nq, dtype):
    """Keys whose every logit is -inf are as keys that are not there, whatever
    their values; rows with no other logit are as rows that see no key."""
    nk, d = 384, 64
    q, k, v = normal(1, nq, 1, d, dtype=dtype), normal(2, nk, 1, d, dtype=dtype), normal(3, nk, 1, d, dtype=dtype)
    q[..., 0] = q[..., 0].abs() + 1
    far = torch.arange(nk, device="cuda") % 16 >= 6
    k[far, :, 0] = -math.inf
    v[far] = 60000.0 if dtype == FP else 3e38
    O, lse = ig.prompt_attention(q, k, v, cu([nq]), cu([nk]), causal=False)
    near = ~far
    o, l, _, tol, tol_l, _ = attend(q[:, 0], k[near, 0], v[near, 0], d ** -0.5)
    within(O[:, 0], o, tol, "O")
    within(lse[0], l, tol_l, "lse")
    k[..., 0] = -math.inf
    O, lse = ig.prompt_attention(q, k, v, cu([nq]), cu([nk]), causal=False)
    assert (O == 0).all() and (lse == -math.inf).all()
    w = ig.key_weights(q, k, torch.zeros_like(lse), cu([nq]), cu([nk]), torch.zeros(1, nk, device="cuda"), causal=False)
    assert (w == 0).all()


def test_logits_far_below_the_largest_weigh_what_they_should():
    # weights of 2^-187 times values of 3e38 are nothing; 2^-126 of them would be 3.5
    nq, nk, d = 256, 256, 64
    q, k, v = torch.zeros(nq, 1, d, dtype=BF, device="cuda"), torch.zeros(nk, 1, d, dtype=BF, device="cuda"), normal(3, nk, 1, d)
    q[..., 0], k[1:, 0, 0], v[1:] = 1.0, -130.0, 3e38
    O, lse = ig.prompt_attention(q, k, v, cu([nq]), cu([nk]), causal=False, softmax_scale=1.0)
    assert torch.equal(O, v[:1].expand(nq, 1, d)) and (lse == 0).all()


@pytest.mark.parametrize("keep", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("P,cap", [(0, 70), (70, 0), (1, 1), (3000, 5), (3000, 3000), (30000, 5)])
def test_a_nan_query_shows_in_its_step(P, cap, keep):
    """Every logit of the row is NaN, in whichever part its keys are."""
    B, Hq, Hkv, d = 40, 4, 2, 64
    q, kp, kc = normal(1, B, Hq, d), normal(2, Hkv, P, d), normal(4, B, Hkv, cap, d)
    lens = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    q[3, 1, 7] = math.nan
    w = torch.zeros(B, Hkv, cap, device="cuda") if keep else None
    O, lse = ig.prefix_attention(q, kp, kp, kc, kc, lens, weights=w)
    bad = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
    bad[3, 1] = True
    nan_rows(lse, bad, "lse")
    nan_rows(O, bad[..., None].expand(B, Hq, d), "O")
    if keep:
        bad = torch.zeros(B, Hkv, cap, dtype=torch.bool, device="cuda")
        bad[3, 0] = True
        nan_rows(w, bad, "weights")


@pytest.mark.parametrize("P", [0, 100])
def test_a_step_whose_logits_are_all_minus_infinity_adds_no_weight(P):
    B, Hq, Hkv, d, cap = 3, 4, 2, 64, 90
    q, kp, kc = normal(1, B, Hq, d).abs() + 1, normal(2, Hkv, P, d), normal(4, B, Hkv, cap, d)
    kp[..., 0], kc[..., 0] = -math.inf, -math.inf
    lens = torch.tensor([90, 33, 0], dtype=torch.int32, device="cuda")
    w = torch.full((B, Hkv, cap), 2.0, device="cuda")
    O, lse = ig.prefix_attention(q, kp, kp.abs().nan_to_num(posinf=1), kc, kc.abs().nan_to_num(posinf=1), lens, weights=w)
    assert (O == 0).all() and (lse == -math.inf).all() and (w == 2).all()


# Keys whose weights are small beside the largest: fp16's steps are 2^-24 from
# 2^-14 down, so the weights are multiplied into its range before they are
# rounded.  The largest is at least 2^7 there, so that a weight is off by at
# most half a step or by 2^-25 / 2^7 of the largest: no more than
#   u |O| + (u + 2 |dx| + 2^-19) sum_j p_j |v_j| + 2^-32 max_j p_j sum_j |v_j|.
def tail_check(O, x, v, dx):
    p = torch.softmax(x, -1)
    o, u = p @ v, 2.0 ** -11
    tol = u * o.abs() + (u + 2 * dx[:, None] + 2.0 ** -19) * (p @ v.abs()) + 2.0 ** -32 * v.abs().sum(0)
    within(O, o, tol, "O")


@pytest.mark.parametrize("sink", [0, 999, 3999])
@pytest.mark.parametrize("nq", [60, 250])
def test_fp16_small_weights_of_a_prompt(nq, sink):
    """One key of weight near 1 and 3999 of 2^-18 to 2^-22 of it, which make up to 1.5% of the sum."""
    nk, d = 4000, 64
    q, k, v = (torch.zeros(n, 1, d, dtype=FP, device="cuda") for n in (nq, nk, nk))
    q[:, 0, 0] = 12.5 + 2.75 * torch.arange(nq, device="cuda") / nq
    k[sink, 0, 0] = 1.0
    v[:] = 1.0
    v[sink] = 0.0
    O, _ = ig.prompt_attention(q, k, v, cu([nq]), cu([nk]), causal=False, softmax_scale=1.0)
    x = q[:, 0].double() @ k[:, 0].double().t()
    tail_check(O[:, 0], x, v[:, 0].double(), d * 2.0 ** -23 * x.abs().amax(1))


@pytest.mark.parametrize("B,P,n", [(1, 0, 4000), (3, 1500, 2500), (2, 4000, 0), (60, 4000, 3)])
def test_fp16_small_weights_of_a_step(B, P, n):
    Hq, d = 8, 64
    q = torch.zeros(B, Hq, d, dtype=FP, device="cuda")
    q[..., 0] = 12.5 + 2.75 * torch.arange(B * Hq, device="cuda").view(B, Hq) / (B * Hq)
    k, v = torch.zeros(1, P + n, d, dtype=FP, device="cuda"), torch.ones(1, P + n, d, dtype=FP, device="cuda")
    k[0, 77, 0], v[0, 77] = 1.0, 0.0
    kc, vc = (t[:, P:].expand(B, 1, n, d).contiguous() for t in (k, v))
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    O, _ = ig.prefix_attention(q, k[:, :P].contiguous(), v[:, :P].contiguous(), kc, vc, lens, softmax_scale=1.0)
    x = q.flatten(0, 1).double() @ k[0].double().t()
    tail_check(O.flatten(0, 1), x, v[0].double(), d * 2.0 ** -23 * x.abs().amax(1))


def test_one_layer_of_odd_sized_lse_and_weights():
    qs, Hq, Hkv, d = [33, 20], 3, 1, 64
    q, k, v = normal(1, 53, Hq, d), normal(2, 53, Hkv, d), normal(3, 53, Hkv, d)
    lse, w = torch.zeros(3, Hq, 53, device="cuda"), torch.zeros(3, Hkv, 53, device="cuda")
    O, _ = ig.prompt_attention(q, k, v, cu(qs), cu(qs), lse=lse[1])
    ig.key_weights(q, k, lse[1], cu(qs), cu(qs), w[1])
    check_prompt(q, k, v, qs, qs, True, O, lse[1], weights=w[1], before=torch.zeros(Hkv, 53, device="cuda"))
    s = step_inputs("odd", BF)
    B, Hkv, cap = s[3].shape[:3]
    lse, w = torch.zeros(3, B, s[0].shape[1], device="cuda"), torch.zeros(3, B, Hkv, cap, device="cuda")
    O, _ = ig.prefix_attention(*s, lse=lse[1], weights=w[1])
    check_step(*s, O, lse[1], torch.zeros_like(w[1]), w[1])
    assert (lse[0] == 0).all() and (lse[2] == 0).all() and (w[0] == 0).all() and (w[2] == 0).all()
    ig.device_status()


def test_evict_caches_without_slots():
    B, Hkv, d = 3, 2, 64
    t = evict_inputs(B, Hkv, 0, d, [0] * B, "spread")
    out = tuple(torch.full((B, Hkv, 5, *x.shape[3:]), 9, dtype=x.dtype, device="cuda") for x in t[:4]) + (
        torch.full((B,), 9, dtype=torch.int32, device="cuda"),)
    got = ig.evict(*t, 5, 1, out=out)
    assert (got[4] == 0).all() and all((x == 9).all() for x in got[:4])
    ig.device_status()


# -------------------------------------- forms that only some sizes reach
def check_evict_long(before, after, budget, recent):
    """check_evict for one long cache, by sorting."""
    k, v, w, pos, lens = before
    n = int(lens[0])
    x, t = w[0, 0, :n].double().cpu().numpy(), pos[0, 0, :n].cpu().numpy().astype(np.int64)
    nan = np.isnan(x)
    order = np.lexsort((np.arange(n), -np.where(nan, 0.0, x), nan, ~(t > t.max() - recent)))
    kept = np.sort(order[:budget])
    source = np.arange(budget)
    stays = np.zeros(budget, dtype=bool)
    stays[kept[kept < budget]] = True
    source[~stays] = kept[kept >= budget]
    at = torch.tensor(source, device="cuda")
    assert int(after[4][0]) == budget
    for got, ref in zip(after[:4], before[:4]):
        assert torch.equal(torch.nan_to_num(got[0, 0, :budget].float()), torch.nan_to_num(ref[0, 0, at].float()))


@pytest.mark.parametrize("place", [True, False], ids=["in_place", "copy"])
@pytest.mark.parametrize("kind", ["ties", "odd"])
@pytest.mark.parametrize("cap,n,budget,recent", [
    (420000, 419999, 100000, 1000),  # a CTA's part of 52512 slots: read again in every pass
    (420000, 300001, 70, 100),
    (80003, 80000, 40000, 7),        # parts of 10016 slots: more than a thread's registers hold
], ids=["unheld", "unheld_recent", "held"])
def test_evict_long_parts(cap, n, budget, recent, kind, place):
    t = evict_inputs(1, 1, cap, 64, [n], kind)
    before = [x.clone() for x in t]
    out = None if place else tuple(
        torch.zeros(1, 1, budget, *x.shape[3:], dtype=x.dtype, device="cuda") for x in t[:4]) + (t[4].clone(),)
    check_evict_long(before, ig.evict(*t, budget, recent, out=out), budget, recent)
    ig.device_status()


@pytest.mark.parametrize("kind", ["ties", "odd"])
@pytest.mark.parametrize("Hkv,cap,n", [(2, 2050, 2049), (2, 4000, 3999), (1, 6001, 6000), (80, 5000, 4900)])
def test_evict_clusters_of_two_and_four(Hkv, cap, n, kind):
    t = evict_inputs(1, Hkv, cap, 64, [n], kind)
    before = [x.clone() for x in t]
    check_evict(before, ig.evict(*t, n // 3, 100), n // 3, 100)
    ig.device_status()


@pytest.mark.parametrize("keep", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("B,P,lens,cap", [(1, 0, [49000], 50000), (1, 17000, [49000], 50000), (1, 40000, [0], 0),
                                          (2, 300, [66000, 40000], 66000)])
def test_steps_with_more_than_32_parts(B, P, lens, cap, keep):
    Hq, Hkv, d = 4, 1, 64
    q, kp, vp = normal(1, B, Hq, d, scale=1.2), normal(2, Hkv, P, d, scale=1.2), normal(3, Hkv, P, d)
    kc, vc = normal(4, B, Hkv, cap, d, scale=1.2), normal(5, B, Hkv, cap, d)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = normal(6, B, Hkv, cap, dtype=torch.float32).abs()
    w = before.clone() if keep else None
    O, lse = ig.prefix_attention(q, kp, vp, kc, vc, n, weights=w)
    check_step(q, kp, vp, kc, vc, n, O, lse, before, w)
    ig.device_status()


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_prompt_among_short_ones(d):
    qs, ks = [1 + i % 5 for i in range(30)] + [700, 2], [3 + i % 7 for i in range(30)] + [6000, 2]
    q, k, v = normal(1, sum(qs), 4, d, scale=1.2), normal(2, sum(ks), 2, d, scale=1.2), normal(3, sum(ks), 2, d)
    O, lse = ig.prompt_attention(q, k, v, cu(qs), cu(ks))
    w = ig.key_weights(q, k, lse, cu(qs), cu(ks), torch.zeros(2, sum(ks), device="cuda"))
    check_prompt(q, k, v, qs, ks, True, O, lse, weights=w, before=torch.zeros_like(w))
    ig.device_status()


def test_the_readme_example():
    """The language-model example of README.md, each step against its definition."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = text.split("```python\n")[1].split("```")[0]
    qs, Hq, Hkv, d = [1500, 40, 1100], 4, 2, 64
    B, T, c = len(qs), sum(qs), cu(qs)
    q, k, v = normal(1, T, Hq, d), normal(2, T, Hkv, d), normal(3, T, Hkv, d)
    env = dict(q=q, k=k, v=v, cu=c, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, q1=normal(4, B, Hq, d),
               k_shared=normal(5, Hkv, 300, d), v_shared=normal(6, Hkv, 300, d))
    head, tail = code.split("# keep 1024 keys")
    exec(head, env)
    check_prompt(q, k, v, qs, qs, True, env["o"], env["lse"], weights=env["w"], before=torch.zeros(Hkv, T, device="cuda"))
    start = 0
    for b, n in enumerate(qs):
        assert torch.equal(env["kc"][b, :, :n], k[start:start + n].transpose(0, 1))
        assert torch.equal(env["vc"][b, :, :n], v[start:start + n].transpose(0, 1))
        assert torch.equal(env["wc"][b, :, :n], env["w"][:, start:start + n])
        start += n
    before = [env[n] for n in ("kc", "vc", "wc", "pos", "lens")]
    exec("# keep 1024 keys" + tail.split("# one token")[0], env)
    after = [env[n] for n in ("kc", "vc", "wc", "pos", "lens")]
    check_evict(before, after, 1024, 128)
    weights = env["wc"].clone()
    exec("# one token" + tail.split("# one token")[1], env)
    check_step(env["q1"], env["k_shared"], env["v_shared"], after[0], after[1], after[4], env["o"], env["lse"], weights,
               env["wc"])
    ig.device_status()


# ----------------------------------------------------------------- refusals
def test_binding_refusals():
    q, k = normal(1, 8, 4, 64), normal(2, 8, 2, 64)
    c = cu([8])
    for err, args in [
        (TypeError, (q.float(), k, k, c, c)), (TypeError, (q, k.half(), k, c, c)), (TypeError, (q, k, None, c, c)),
        (ValueError, (q, k[:, :, :32], k, c, c)), (ValueError, (q, k, k[:5], c, c)),
        (ValueError, (q[:, :3], k, k, c, c)), (TypeError, (q, k, k, c.long(), c)),
        (ValueError, (q, k, k, c, cu([4, 4]))), (ValueError, (q, k, k, c[:1], c[:1])),
        (ValueError, (q, k[:, :1].expand(8, 2, 64), k, c, c)),          # rows that overlap
        (ValueError, (q.transpose(1, 2), k, k, c, c)),
        (ValueError, (normal(1, 8, 4, 68)[..., :64], k, k, c, c)),      # stride not of 16 bytes
        (ig.InstaGenError, (q[..., :32].contiguous(), k[..., :32].contiguous(), k[..., :32].contiguous(), c, c)),
        (ig.InstaGenError, (normal(1, 8, 4, 72)[..., 4:68], k, k, c, c)),  # address not of 16 bytes
        (ig.InstaGenError, (q.cpu(), k, k, c, c)), (ig.InstaGenError, (q, k, k, c.cpu(), c)),
    ]:
        with pytest.raises(err):
            ig.prompt_attention(*args)
    with pytest.raises(ig.InstaGenError):
        ig.prompt_attention(q, k, k, c, c, softmax_scale=0.0)
    with pytest.raises(ig.InstaGenError, match="workspace"):
        ig.prompt_attention(q, k, k, c, c, workspace=torch.empty(8, device="cuda"))
    s = step_inputs("tiles", BF)
    w = torch.zeros(s[3].shape[:3], device="cuda")
    for err, i, x in [(TypeError, 0, s[0].half()), (ValueError, 0, s[0][:3]), (ValueError, 1, s[1][:2]),
                      (ValueError, 2, s[2][:, :9]), (ValueError, 1, None), (ValueError, 4, s[4][:, :1]),
                      (TypeError, 5, s[5].long()), (ValueError, 5, s[5][:2]), (ValueError, 0, s[0][:, :7])]:
        with pytest.raises(err):
            ig.prefix_attention(*(x if j == i else t for j, t in enumerate(s)))
    with pytest.raises(ValueError):
        ig.prefix_attention(*s, weights=w[:, :, :5].contiguous())
    e = evict_inputs(2, 2, 50, 64, [50, 20], "spread")
    for budget, recent in ((0, 0), (51, 0), (10, -1)):
        with pytest.raises(ValueError):
            ig.evict(*e, budget, recent)
    with pytest.raises(ValueError):
        ig.evict(e[0], e[1], e[2], e[3][:, :1].contiguous(), e[4], 10, 0)
    other = [t[:, :, :20].contiguous() if t.dim() > 1 else t.clone() for t in e]
    with pytest.raises(ig.InstaGenError):  # some outputs the inputs, some not
        ig.evict(*e, 10, 0, out=(other[0], other[1], other[2], other[3], e[4]))
    ig.device_status()
