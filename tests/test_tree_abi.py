"""Host-side checks of the tree calls (no GPU needed): sizes, the rotary table, and refusals before any
launch.  Addresses are made up; no call here reaches a launch."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_81_b200 import build, gdn

INVALID, UNSUPPORTED, MISALIGNED, ALIAS, WORKSPACE = 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def fake_inputs(H_k=2, H_v=6):
    s = gdn.GdnInputs()
    for i, f in enumerate(("q", "k", "v", "a", "b", "z", "conv_w", "A_log", "norm_w")):
        setattr(s, f, (i + 1) << 32)
    s.stride_q = s.stride_k = H_k * 128
    s.stride_v = s.stride_z = H_v * 128
    s.stride_a = s.stride_b = H_v
    s.H_k, s.H_v, s.scale = H_k, H_v, 1.0
    return s


STATE, CONV, OUT, PARENT, ACC, SLOT = (x << 36 for x in range(1, 7))


def decode_tree(lib, inp=None, N=2, T=4, parent=PARENT, state=STATE, conv=CONV, slot=None, slots=2, out=OUT):
    return lib.gdn_decode_tree(ctypes.byref(inp or fake_inputs()), N, T, parent, state, conv, slot, slots, out, None, None)


def test_decode_tree_refusals(lib):
    assert decode_tree(lib, N=0) == 0
    assert decode_tree(lib, N=-1) == INVALID
    assert decode_tree(lib, T=0) == INVALID
    assert decode_tree(lib, T=65) == INVALID
    assert decode_tree(lib, N=65536, slots=65536) == UNSUPPORTED
    assert decode_tree(lib, slots=1) == INVALID          # slot n for sequence n needs N slots
    assert decode_tree(lib, state=None) == INVALID
    assert decode_tree(lib, out=None) == INVALID
    assert decode_tree(lib, state=STATE + 4) == MISALIGNED
    assert decode_tree(lib, parent=PARENT + 2) == MISALIGNED
    assert decode_tree(lib, out=STATE + 64) == ALIAS
    assert decode_tree(lib, out=CONV) == ALIAS
    assert decode_tree(lib, out=PARENT) == ALIAS
    inp = fake_inputs()
    assert decode_tree(lib, inp, out=inp.v) == ALIAS
    assert decode_tree(lib, inp, out=inp.conv_w) == ALIAS
    inp.stride_q = 100
    assert decode_tree(lib, inp) == INVALID
    assert decode_tree(lib, fake_inputs(1, 9)) == UNSUPPORTED


def commit(lib, inp=None, N=2, T=4, parent=PARENT, acc=ACC, s_in=STATE, s_out=STATE, c_in=CONV, c_out=CONV, slots=2):
    return lib.gdn_decode_tree_commit(ctypes.byref(inp or fake_inputs()), N, T, parent, acc, s_in, s_out, c_in, c_out,
                                      None, slots, None, None)


def test_decode_tree_commit_refusals(lib):
    assert commit(lib, N=0) == 0
    assert commit(lib, acc=None) == INVALID
    assert commit(lib, s_out=None) == INVALID
    assert commit(lib, T=65) == INVALID
    assert commit(lib, s_out=STATE + 65536) == ALIAS     # neither in place nor apart
    assert commit(lib, c_out=CONV + 16) == ALIAS
    assert commit(lib, c_out=STATE) == ALIAS
    assert commit(lib, s_out=ACC) == ALIAS
    assert commit(lib, s_out=fake_inputs().q) == ALIAS
    assert commit(lib, c_in=CONV + 8, c_out=CONV + 8) == MISALIGNED


def test_header_says_what_the_commit_reads():
    """Every raw row of the path becomes conv state, q's too: the contract may not let a caller reuse q before the commit."""
    with open(os.path.join(build.INCLUDE, "gdn.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    doc = text[text.index("The commit of gdn_decode_tree:"):text.index("gdn_status gdn_decode_tree_commit(")]
    assert "q and z are not read" not in doc
    assert "last raw rows of q, k and v become the conv state" in doc


def test_header_bounds_a_bf16_rounding():
    """A rounding to bf16 is off by up to 2^-8 of the value, not 2^-9: the header's bound for attention's probabilities."""
    x = torch.linspace(1, 2, 100001, dtype=torch.float64)
    off = float(((x.to(torch.bfloat16).double() - x).abs() / x).max())
    assert 2.0 ** -9 < off <= 2.0 ** -8
    with open(os.path.join(build.INCLUDE, "gdn.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    doc = text[text.index("Attention of a tree's nodes over a KV cache"):text.index("size_t gdn_attention_tree_workspace_size(")]
    assert "2^-9" not in doc and "(relative error <= 2^-8 each" in doc


def attention(lib, H=24, Hkv=4, D=256, scale=0.0625, N=2, T=4, cap=100, ld_q=None, ld_kt=None, out=OUT, ws=7 << 36, nb=None,
              k=8 << 36, v=9 << 36, g=None, ld_g=0, q=10 << 36, ln=11 << 36):
    nb = lib.gdn_attention_tree_workspace_size(H, Hkv, D, N, T) if nb is None else nb
    return lib.gdn_attention_tree(q, H * D if ld_q is None else ld_q, 12 << 36, Hkv * D if ld_kt is None else ld_kt, 13 << 36, Hkv * D,
                                  k, v, cap, ln, PARENT, g, ld_g, H, Hkv, D, scale, N, T, out, ws, nb, None, None)


def test_attention_tree_refusals(lib):
    assert attention(lib, N=0) == 0
    assert attention(lib, D=64) == UNSUPPORTED
    assert attention(lib, H=68, Hkv=4) == UNSUPPORTED
    assert attention(lib, H=25) == INVALID
    assert attention(lib, T=65) == INVALID
    assert attention(lib, cap=0) == INVALID
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert attention(lib, scale=scale) == INVALID
    assert attention(lib, ld_q=24 * 256 - 8) == INVALID
    assert attention(lib, ld_q=24 * 256 + 4) == MISALIGNED
    assert attention(lib, k=(8 << 36) + 8) == MISALIGNED
    assert attention(lib, g=14 << 36, ld_g=100) == INVALID
    assert attention(lib, ln=None) == INVALID
    assert attention(lib, nb=0) == WORKSPACE
    assert attention(lib, ws=None) == WORKSPACE
    assert attention(lib, out=8 << 36) == ALIAS
    assert attention(lib, out=10 << 36) == ALIAS
    assert attention(lib, ws=8 << 36) == ALIAS
    assert attention(lib, out=7 << 36) == ALIAS
    assert lib.gdn_attention_tree_workspace_size(24, 4, 64, 1, 1) == 0
    assert lib.gdn_attention_tree_workspace_size(24, 5, 256, 1, 1) == 0
    assert lib.gdn_attention_tree_workspace_size(24, 4, 256, 1, 65) == 0


def append(lib, k=8 << 36, v=9 << 36, ln=11 << 36, lo=11 << 36, kt=12 << 36, D=256, cap=50, N=2, acc=ACC, ld=4 * 256):
    return lib.gdn_attn_tree_commit(kt, ld, 13 << 36, 4 * 256, 4, D, N, 4, PARENT, acc, k, v, cap, ln, lo, None, None)


def test_attn_tree_commit_refusals(lib):
    assert append(lib, N=0) == 0
    assert append(lib, acc=None) == INVALID
    assert append(lib, cap=0) == INVALID
    assert append(lib, ld=8) == INVALID
    assert append(lib, D=96) == UNSUPPORTED
    assert append(lib, v=8 << 36) == ALIAS
    assert append(lib, kt=8 << 36) == ALIAS
    assert append(lib, lo=(11 << 36) + 4) == ALIAS
    assert append(lib, lo=8 << 36) == ALIAS
    assert append(lib, k=(8 << 36) + 2) == MISALIGNED


def rope_call(lib, rope=None, n=4, H=2, Hkv=1, q=1 << 36, ld_q=256, k=2 << 36, ld_k=128, v=3 << 36, ld_v=128, rows=None, n_rows=4,
              qo=4 << 36, ld_qo=256, ko=5 << 36, ld_ko=128, vo=6 << 36, ld_vo=128):
    rope = rope or gdn.make_rope(128, 64)
    return lib.gdn_qk_norm_rope(ctypes.byref(rope), n, H, Hkv, q, ld_q, k, ld_k, v, ld_v, None, None, None, rows, n_rows, qo, ld_qo,
                                ko, ld_ko, vo, ld_vo, None, None)


def test_qk_norm_rope_refusals(lib):
    assert rope_call(lib, n=0) == 0
    assert rope_call(lib, H=0, Hkv=0, q=None, k=None, v=None, vo=None) == 0
    assert rope_call(lib, gdn.GdnRope()) == INVALID      # never initialised
    assert rope_call(lib, n=-1) == INVALID
    assert rope_call(lib, q=None) == INVALID
    assert rope_call(lib, v=None) == INVALID             # v_out without v
    assert rope_call(lib, n_rows=3) == INVALID           # row t for token t needs n_tok rows
    assert rope_call(lib, ld_q=128) == INVALID
    assert rope_call(lib, ld_k=132) == MISALIGNED
    assert rope_call(lib, qo=(4 << 36) + 2) == MISALIGNED
    assert rope_call(lib, n=2 ** 31, n_rows=2 ** 31) == UNSUPPORTED
    assert rope_call(lib, qo=(1 << 36) + 16) == ALIAS    # overlapping, not in place
    assert rope_call(lib, ko=2 << 36, rows=7 << 36) == ALIAS  # in place under a permutation
    assert rope_call(lib, vo=3 << 36) == ALIAS
    assert rope_call(lib, vo=5 << 36) == ALIAS


def test_rope_init(lib):
    def init(D=128, R=128, layout=0, scaling=0, base=1e4, factor=1.0, orig=0, fast=32.0, slow=1.0, eps=1e-6):
        rope = gdn.GdnRope()
        return lib.gdn_rope_init(ctypes.byref(rope), D, R, layout, scaling, base, factor, orig, fast, slow, eps), rope
    assert init()[0] == 0
    assert init(D=130)[0] == UNSUPPORTED
    assert init(D=512, R=64)[0] == UNSUPPORTED
    assert init(R=72)[0] == UNSUPPORTED
    assert init(R=144)[0] == INVALID
    assert init(layout=2)[0] == INVALID
    assert init(scaling=4)[0] == INVALID
    assert init(base=1.0)[0] == INVALID
    assert init(factor=0.5)[0] == INVALID
    assert init(factor=math.inf)[0] == INVALID
    assert init(eps=-1.0)[0] == INVALID
    assert init(scaling=3, factor=4.0)[0] == INVALID     # no original length
    assert init(scaling=3, factor=4.0, orig=4096, fast=1.0)[0] == INVALID
    with pytest.raises(ValueError):
        gdn.make_rope(128, scaling="cubic")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("R", [16, 64, 256])
def test_rope_table(lib, scaling, R):
    """turns[i] / 2^64 is theta_i / 2 pi, to the rounding of the oracle's 64-bit frequency."""
    kw = dict(scaling=scaling, factor=4.0, original_len=4096)
    rope = gdn.make_rope(256, R, base=1e6, **kw)
    theta, amp = oracle.tree.rope_frequencies(R, 1e6, **kw)
    got = np.array([rope.turns[i] for i in range(R // 2)], dtype=np.float64) / 2.0 ** 64 * (2 * math.pi)
    np.testing.assert_allclose(got, theta, rtol=1e-14, atol=2.0 ** -62)
    assert rope.amplitude == np.float32(amp)
    assert all(rope.turns[i] == 0 for i in range(R // 2, 128))


def test_yarn_ramp_past_the_last_pair(lib):
    """The pair that turns once lies beyond the last one: the ramp ends there, not at the last pair.  Numbers written out."""
    # 8 pairs, base 10^4: 16 ln(32768 / 2 pi 32) / 2 ln 10^4 = 4.42, 16 ln(32768 / 2 pi) / 2 ln 10^4 = 7.43: from 4 to 8
    kw = dict(base=1e4, scaling="yarn", factor=8.0, original_len=32768)
    want = [1, 10 ** -0.5, 10 ** -1, 10 ** -1.5, 10 ** -2,
            10 ** -2.5 * (0.75 + 0.25 / 8), 10 ** -3 * (0.5 + 0.5 / 8), 10 ** -3.5 * (0.25 + 0.75 / 8)]
    rope = gdn.make_rope(64, 16, **kw)
    np.testing.assert_allclose([rope.turns[i] / 2.0 ** 64 * 2 * math.pi for i in range(8)], want, rtol=1e-13)
    np.testing.assert_allclose(oracle.tree.rope_frequencies(16, **kw)[0], want, rtol=1e-13)
    # 64 pairs at 131,072 positions: 45.03 and 69.11, so from 45 to 70; the last pair, 63, at 18 / 25
    kw = dict(base=1e4, scaling="yarn", factor=16.0, original_len=131072)
    rope = gdn.make_rope(128, **kw)
    for i, ramp in ((45, 0.0), (50, 0.2), (55, 0.4), (63, 0.72)):
        want = 10 ** (-4 * i / 64) * (1 - ramp + ramp / 16)
        assert rope.turns[i] / 2.0 ** 64 * 2 * math.pi == pytest.approx(want, rel=1e-13)
        assert oracle.tree.rope_frequencies(128, **kw)[0][i] == pytest.approx(want, rel=1e-13)


def test_layer_tree_sizes_and_refusals(lib):
    assert lib.gdn_layer_tree_workspace_size(16, 48, 2, 65) == 0
    assert lib.gdn_layer_tree_workspace_size(16, 48, 1, 64) >= 64 * (16480 + 6144) * 2
    assert lib.gdn_attn_layer_tree_workspace_size(1, 0) == 0
    need = lib.gdn_layer_tree_workspace_size(2, 6, 2, 4)
    L = gdn.GdnLayer()
    for i, f in enumerate(("w_in", "w_out", "conv_w", "A_log", "norm_w")):
        setattr(L, f, (i + 20) << 36)
    L.ld_w_in, L.ld_w_out, L.H_k, L.H_v, L.hidden, L.scale = 128, 768, 2, 6, 128, 1.0

    def call(x=30 << 36, y=31 << 36, ws=32 << 36, nb=need, T=4, ldy=128, state=STATE):
        return lib.gdn_layer_decode_tree(ctypes.byref(L), 2, T, PARENT, x, 128, state, CONV, None, 2, y, ldy, ws, nb, None, None)
    assert call(T=65) == INVALID
    assert call(x=None) == INVALID
    assert call(nb=need - 1) == WORKSPACE
    assert call(ldy=64) == INVALID
    assert call(y=32 << 36) == ALIAS
    assert call(y=STATE) == ALIAS
    assert call(state=32 << 36) == ALIAS
    assert call(x=(30 << 36) + 2) == MISALIGNED
    L.hidden = 100
    assert call() == UNSUPPORTED
    L.hidden = 128
    assert lib.gdn_layer_tree_commit(ctypes.byref(L), 2, 4, PARENT, ACC, 32 << 36, CONV, None, 2, 32 << 36, need, None, None) == ALIAS
    assert lib.gdn_layer_tree_commit(ctypes.byref(L), 2, 4, PARENT, ACC, STATE, CONV, None, 2, 32 << 36, 5, None, None) == WORKSPACE
    assert lib.gdn_attn_layer_tree_commit(2, 4, PARENT, ACC, STATE, CONV, 9, SLOT, 32 << 36, 5, None, None) == WORKSPACE


def cpu_layer(hidden=64, H_k=1, H_v=2):
    L = gdn.GdnLayer()
    L.H_k, L.H_v, L.hidden = H_k, H_v, hidden
    return L


def cpu_pool(slots, H_k=1, H_v=2):
    return torch.zeros(slots, H_v, 128, 128), torch.zeros(slots, 3, (2 * H_k + H_v) * 128, dtype=torch.bfloat16)


def test_layer_calls_refuse_a_pool_of_fewer_slots_than_sequences(lib):
    """Without state_slot sequence n reads (and at the commit writes) slot n."""
    L, N, T = cpu_layer(), 3, 2
    x, ws = torch.zeros(N * T, 64, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8)
    acc = torch.zeros(N, dtype=torch.int32)
    with pytest.raises(ValueError, match="slots"):
        gdn.layer_decode_tree(L, N, T, None, x, *cpu_pool(2), ws)
    with pytest.raises(ValueError, match="slots"):
        gdn.layer_tree_commit(L, N, T, None, acc, *cpu_pool(2), ws)


def bf(*shape, device="cpu"):
    return torch.zeros(*shape, dtype=torch.bfloat16, device=device)


BAD_X = [  # of the wrong type, on another device, too few rows, too narrow, transposed, of another rank
    (torch.zeros(6, 64), TypeError), (bf(6, 64, device="meta"), ValueError), (bf(5, 64), ValueError), (bf(6, 63), ValueError),
    (bf(64, 6).T, ValueError), (bf(6 * 64), ValueError)]


@pytest.mark.parametrize("bad,error", BAD_X, ids=["fp32", "device", "rows", "width", "transposed", "rank"])
@pytest.mark.parametrize("name", ["x", "y"])
@pytest.mark.parametrize("attn", [False, True])
def test_layer_calls_check_their_matrices(lib, bad, error, name, attn):
    L, N, T = cpu_layer(), 3, 2
    m = {"x": bf(6, 64), "y": bf(6, 64), name: bad}
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(error, match=name):
        if attn:
            gdn.attn_layer_decode_tree(L, N, T, None, m["x"], bf(N, 5, 4, 256), bf(N, 5, 4, 256), torch.zeros(N, dtype=torch.int32), ws,
                                       y=m["y"])
        else:
            gdn.layer_decode_tree(L, N, T, None, m["x"], *cpu_pool(N), ws, y=m["y"])


BAD_WS = [torch.zeros(1 << 16, dtype=torch.uint8, device="meta"), torch.zeros(2, 1 << 16, dtype=torch.uint8)[:, ::2]]
BAD_ERR = [torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32, device="meta"), torch.zeros(0, dtype=torch.int32)]


@pytest.mark.parametrize("what,bad", [("workspace", w) for w in BAD_WS] + [("err", e) for e in BAD_ERR])
def test_tree_calls_check_their_workspace_and_error_word(lib, what, bad):
    L, N, T = cpu_layer(), 1, 2
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws, err = (bad, None) if what == "workspace" else (torch.zeros(1 << 16, dtype=torch.uint8), bad)
    S, C = cpu_pool(N)
    kc, vc, n = bf(N, 5, 4, 256), bf(N, 5, 4, 256), i32(N)
    kt = bf(N * T, 4, 256)
    calls = [lambda: gdn.layer_decode_tree(L, N, T, None, bf(2, 64), S, C, ws, err=err),
             lambda: gdn.layer_tree_commit(L, N, T, None, i32(N), S, C, ws, err=err),
             lambda: gdn.attn_layer_decode_tree(L, N, T, None, bf(2, 64), kc, vc, n, ws, err=err),
             lambda: gdn.attn_layer_tree_commit(N, T, None, i32(N), kc, vc, n, ws, err=err),
             lambda: gdn.attention_tree(bf(2, 24, 256), kt, kt, kc, vc, n, T=T, workspace=ws, err=err)]
    if what == "err":
        inp = fake_inputs(1, 2)
        calls += [lambda: gdn.decode_tree(inp, N, T, None, S, C, err=err),
                  lambda: gdn.decode_tree_commit(inp, N, T, None, i32(N), S, C, err=err),
                  lambda: gdn.qk_norm_rope(gdn.make_rope(256), kt, err=err),
                  lambda: gdn.attn_tree_commit(kt, kt, T, None, i32(N), kc, vc, n, err=err)]
    for call in calls:
        with pytest.raises(ValueError, match=what):
            call()


def cpu_inputs(tokens, H_k=1, H_v=2, short=None, away=None):
    """A descriptor of CPU tensors; one may hold fewer tokens, one may lie elsewhere."""
    n = {k: tokens - (k == short) for k in ("q", "k", "v", "a", "b", "z")}
    dev = lambda k: "meta" if k == away else "cpu"
    w = {"q": H_k * 128, "k": H_k * 128, "v": H_v * 128, "a": H_v, "b": H_v, "z": H_v * 128}
    return gdn.make_inputs(*(bf(n[k], w[k], device=dev(k)) for k in ("q", "k", "v", "a", "b", "z")),
                           bf((2 * H_k + H_v) * 128, 4, device=dev("conv_w")), torch.zeros(H_v, device=dev("A_log")), bf(128))


@pytest.mark.parametrize("bad,words", [({"short": k}, "5 tokens, not 6") for k in ("q", "v", "a", "z")] +
                         [({"away": k}, "meta") for k in ("k", "b", "conv_w", "A_log")])
def test_decode_tree_calls_check_the_descriptor_s_tensors(lib, bad, words):
    """The descriptor holds addresses alone: how many tokens there are, and where, is kept beside them."""
    inp = cpu_inputs(6, **bad)
    with pytest.raises(ValueError, match=words):
        gdn.decode_tree(inp, 3, 2, None, *cpu_pool(3))
    with pytest.raises(ValueError, match=words):
        gdn.decode_tree_commit(inp, 3, 2, None, torch.zeros(3, dtype=torch.int32), *cpu_pool(3))


def test_layer_tree_calls_check_the_layer_s_device(lib):
    ws, acc = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    L = gdn.make_layer(bf(64 * 16, 64, device="meta"), bf(64, 256), bf(512, 4), torch.zeros(2), bf(128), 1, 2)
    with pytest.raises(ValueError, match="meta"):
        gdn.layer_decode_tree(L, 1, 2, None, bf(2, 64), *cpu_pool(1), ws)
    with pytest.raises(ValueError, match="meta"):
        gdn.layer_tree_commit(L, 1, 2, None, acc, *cpu_pool(1), ws)
    L = gdn.make_attn_layer(bf(gdn.ATTN_N_IN, 64), bf(64, 24 * 256), bf(256), bf(256, device="meta"))
    with pytest.raises(ValueError, match="meta"):
        gdn.attn_layer_decode_tree(L, 1, 2, None, bf(2, 64), bf(1, 5, 4, 256), bf(1, 5, 4, 256), acc, ws)


def test_tree_oracle_paths():
    assert oracle.tree.paths([-1, 0, -1, 1, -2, 4, 2]) == [[0], [0, 1], [2], [0, 1, 3], [], [], [2, 6]]
    assert oracle.tree.paths([0, -1]) == [[], [1]]
