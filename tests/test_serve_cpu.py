"""Host-side checks of the language-model entry points: parameter refusals and
workspace sizes through the C ABI (no call here reaches a kernel)."""
import ctypes

import pytest

import block_sparse_attention_head_b200 as ig
from block_sparse_attention_head_b200 import build as igbuild

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    igbuild.build()
    return ig.lib()


def prompt(**kw):
    d = kw.get("d", 64)
    a = dict(nseq=2, Hq=8, Hkv=2, d=d, Tq=100, Tk=120, dtype=0, causal=1, softmax_scale=0.125, q_tok=8 * d, q_head=d,
             k_tok=2 * d, k_head=d, v_tok=2 * d, v_head=d, o_tok=8 * d, o_head=d)
    a.update(kw)
    return ig.PromptParams(**a)


def cache(**kw):
    a = dict(B=3, Hq=8, Hkv=2, d=64, P=100, cap=50, dtype=1, softmax_scale=0.125, q_seq=512, prefix_head=6400)
    a.update(kw)
    return ig.CacheParams(**a)


def prompt_call(lib, p, Q=FAKE, K=FAKE, V=FAKE, O=FAKE, cu=FAKE, ws=FAKE, n=1 << 40):
    return lib.instagen_prompt_attention(Q, K, V, cu, cu, ctypes.byref(p), O, None, ws, n, None)


def test_struct_sizes(lib):
    assert ctypes.sizeof(ig.PromptParams) == 104 and ig.PromptParams.q_tok.offset == 40
    assert ctypes.sizeof(ig.CacheParams) == 48 and ig.CacheParams.q_seq.offset == 32


def test_packed_blocks_are_the_structs(lib):
    from block_sparse_attention_head_b200 import serve
    a = (3, 8, 2, 64, 100, 120, 1, 0, 0.125, *range(8, 72, 8))
    assert serve._prompt_block(*a) == bytes(ig.PromptParams(*a))
    a = (3, 8, 2, 64, 100, 50, 1, 0.125, 512, 6400)
    assert serve._cache_block(*a) == bytes(ig.CacheParams(*a))


BAD_PROMPTS = [
    (dict(nseq=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(dtype=2), INVALID), (dict(causal=2), INVALID),
    (dict(softmax_scale=0.0), INVALID), (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
    (dict(softmax_scale=float("inf")), INVALID), (dict(q_tok=0), INVALID), (dict(k_tok=60), INVALID),
    (dict(k_head=68), INVALID), (dict(q_head=-64), INVALID), (dict(k_tok=1 << 39), INVALID),
    (dict(nseq=(1 << 20) + 1), UNSUPPORTED), (dict(Tq=2 ** 31 - 1), UNSUPPORTED), (dict(Tk=2 ** 31 - 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_PROMPTS)
def test_prompt_params_refused(lib, kw, code):
    p = prompt(**kw)
    assert lib.instagen_prompt_attention_workspace_size(ctypes.byref(p)) == 0
    assert lib.instagen_key_weights_workspace_size(ctypes.byref(p)) == 0
    assert prompt_call(lib, p) == code
    assert lib.instagen_key_weights(FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(p), FAKE, FAKE, 1 << 40, None) == code


def test_prompt_pointers_refused(lib):
    p = prompt()
    need = lib.instagen_prompt_attention_workspace_size(ctypes.byref(p))
    assert need >= 256 and lib.instagen_key_weights_workspace_size(ctypes.byref(p)) >= 256
    for kw in (dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(cu=None), dict(Q=ODD), dict(K=ODD),
               dict(V=ODD), dict(O=ODD)):
        assert prompt_call(lib, p, **kw) == INVALID
    for kw in (dict(ws=ODD), dict(n=need - 1)):
        assert prompt_call(lib, p, **kw) == WORKSPACE
    split = prompt(nseq=1, Tq=4, Tk=100000)  # few rows, many keys: parts are kept on the side
    need = lib.instagen_prompt_attention_workspace_size(ctypes.byref(split))
    assert need > 256
    for kw in (dict(ws=None), dict(ws=ODD), dict(n=need - 1)):
        assert prompt_call(lib, split, **kw) == WORKSPACE
    for kw in (dict(v_tok=60), dict(v_head=0), dict(o_tok=8), dict(o_head=1)):
        assert prompt_call(lib, prompt(**kw)) == INVALID
    assert lib.instagen_prompt_attention(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, 1 << 40, None) == INVALID
    for i in range(5):
        a = [FAKE] * 5
        a[i] = None
        assert lib.instagen_key_weights(*a, ctypes.byref(p), FAKE, FAKE, 1 << 40, None) == INVALID
    assert lib.instagen_key_weights(*[FAKE] * 5, ctypes.byref(p), None, FAKE, 1 << 40, None) == INVALID
    assert lib.instagen_key_weights(*[FAKE] * 5, ctypes.byref(p), FAKE, FAKE, 16, None) == WORKSPACE
    # nothing to do is fine without buffers
    assert prompt_call(lib, prompt(Tq=0), Q=None, O=None) == 0
    assert lib.instagen_key_weights(None, None, None, None, None, ctypes.byref(prompt(Tk=0)), None, None, 0, None) == 0


BAD_CACHES = [
    (dict(B=0), INVALID), (dict(Hkv=3), INVALID), (dict(d=32), UNSUPPORTED), (dict(P=-1), INVALID), (dict(cap=-1), INVALID),
    (dict(dtype=-1), INVALID), (dict(softmax_scale=0.0), INVALID), (dict(q_seq=500), INVALID), (dict(q_seq=516), INVALID),
    (dict(prefix_head=6392), INVALID), (dict(prefix_head=6404), INVALID), (dict(B=40000), UNSUPPORTED),
    (dict(cap=2 ** 30), UNSUPPORTED), (dict(P=2 ** 31 - 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_params_refused(lib, kw, code):
    p = cache(**kw)
    for keep in (0, 1):
        assert lib.instagen_prefix_attention_workspace_size(ctypes.byref(p), keep) == 0
    assert lib.instagen_prefix_attention(*[FAKE] * 6, ctypes.byref(p), FAKE, None, None, FAKE, 1 << 40, None) == code


def test_prefix_attention_pointers_refused(lib):
    p = cache()
    for i in range(6):
        for bad in (None,) + ((ODD,) if i < 5 else ()):
            a = [FAKE] * 6
            a[i] = bad
            assert lib.instagen_prefix_attention(*a, ctypes.byref(p), FAKE, None, None, FAKE, 1 << 40, None) == INVALID
    assert lib.instagen_prefix_attention(*[FAKE] * 6, ctypes.byref(p), None, None, None, FAKE, 1 << 40, None) == INVALID
    for keep in (None, FAKE):
        need = lib.instagen_prefix_attention_workspace_size(ctypes.byref(p), keep is not None)
        assert need >= 256
        assert lib.instagen_prefix_attention(*[FAKE] * 6, ctypes.byref(p), FAKE, None, keep, FAKE, need - 1, None) == WORKSPACE


def test_evict_refused(lib):
    p = cache(P=0, prefix_head=0)
    need = lib.instagen_evict_workspace_size(ctypes.byref(p), 20)
    assert need >= 256
    assert lib.instagen_evict_workspace_size(ctypes.byref(p), 0) == 0
    out = [ctypes.c_void_p((2 + i) << 20) for i in range(5)]

    def call(ins=(FAKE,) * 5, budget=20, recent=4, outs=out, cap_out=30, n=need, q=p):
        return lib.instagen_evict(*ins, ctypes.byref(q), budget, recent, *outs, cap_out, FAKE, n, None)

    assert call(budget=0) == INVALID and call(budget=31) == INVALID and call(recent=-1) == INVALID
    assert call(n=need - 1) == WORKSPACE
    assert call(q=cache(Hkv=3)) == INVALID and call(q=cache(d=16)) == UNSUPPORTED
    for i in range(5):
        ins, outs = [FAKE] * 5, list(out)
        ins[i] = None
        assert call(ins=ins) == INVALID
        outs[i] = None
        assert call(outs=outs) == INVALID
        outs[i] = FAKE  # one output in place, the others not
        assert call(outs=outs) == INVALID
    assert call(outs=[FAKE] * 5, cap_out=49) == INVALID  # in place keeps the slots
    assert call(cap_out=2 ** 31 - 1, budget=5) == UNSUPPORTED


def test_binding_refuses_cpu_tensors(lib):
    import torch
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    c, n = torch.tensor([0, 8], dtype=torch.int32), torch.tensor([8], dtype=torch.int32)
    kc, w, pos = k[None].transpose(1, 2).contiguous(), torch.zeros(1, 2, 8), torch.zeros(1, 2, 8, dtype=torch.int32)
    for call in (lambda: ig.prompt_attention(q, k, k, c, c), lambda: ig.key_weights(q, k, w, c, c, w),
                 lambda: ig.prefix_attention(q[:1], None, None, kc, kc, n), lambda: ig.evict(kc, kc, w, pos, n, 4, 1)):
        with pytest.raises(ig.InstaGenError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        ig.prompt_attention(None, k, k, c, c)


@pytest.mark.parametrize("kw", [dict(Tq=0), dict(Tk=0), dict(Tq=0, Tk=0), dict()])
@pytest.mark.parametrize("Tk", [1, 4096, 100000])
def test_every_valid_prompt_has_a_workspace_size(lib, Tk, kw):
    p = prompt(nseq=1, Hq=8, Hkv=8, **{"Tk": Tk, "Tq": 4, **kw})
    assert lib.instagen_prompt_attention_workspace_size(ctypes.byref(p)) >= 256
    assert lib.instagen_key_weights_workspace_size(ctypes.byref(p)) >= 256


def test_fp32_buffers_may_start_at_any_element(lib):
    """lse and weights: a layer of a larger buffer.  (The workspace is refused
    here, after every pointer has been accepted.)"""
    four, two = ctypes.c_void_p((1 << 20) + 4), ctypes.c_void_p((1 << 20) + 2)
    split = prompt(nseq=1, Tq=4, Tk=100000)
    for lse, code in ((four, WORKSPACE), (two, INVALID)):
        assert lib.instagen_prompt_attention(*[FAKE] * 5, ctypes.byref(split), FAKE, lse, FAKE, 16, None) == code
        assert lib.instagen_key_weights(FAKE, FAKE, lse, FAKE, FAKE, ctypes.byref(prompt()), FAKE, FAKE, 16, None) == code
        assert lib.instagen_key_weights(FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(prompt()), lse, FAKE, 16, None) == code
        for a in ((lse, None), (None, lse), (lse, lse)):
            assert lib.instagen_prefix_attention(*[FAKE] * 6, ctypes.byref(cache()), FAKE, *a, FAKE, 16, None) == code


def test_evict_takes_caches_without_slots(lib):
    p = cache(P=0, prefix_head=0, cap=0)
    need = lib.instagen_evict_workspace_size(ctypes.byref(p), 20)
    out = [ctypes.c_void_p((2 + i) << 20) for i in range(5)]

    def call(ins, outs=out, n=need - 1):
        return lib.instagen_evict(*ins, ctypes.byref(p), 20, 4, *outs, 30, FAKE, n, None)

    assert need > 0 and call([None] * 4 + [FAKE]) == WORKSPACE  # (only that is refused)
    assert call([None] * 5) == INVALID                          # lens is read
    assert call([None] * 4 + [FAKE], outs=[None] + out[1:]) == INVALID
