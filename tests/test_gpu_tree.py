"""Trees of drafted tokens (through the C ABI) against the fp64 oracle: gdn_decode_tree,
gdn_decode_tree_commit, gdn_attention_tree, gdn_attn_tree_commit, gdn_qk_norm_rope, and the layer
calls made of them.

Tolerances.  The delta-rule mixer is held to the bound of every mixer test (OUT_TOL rms + one bf16
step), its commit to bitwise equality with decoding the path.  gdn_qk_norm_rope: fp32 arithmetic, whose
chain (a sum of at most 256 squares in 13 steps, rsqrtf, three products, sincospif at an argument
rounded to 24 bits, two products and a sum) stays below 2^-18 of |y1| + |y2|, and one rounding to
bf16 (2^-8 relative).  gdn_attention_tree: the probabilities enter as bf16 (2^-8 each, so 2^-8 of sum
p |v|), the scores are D exact products summed in fp32 (each partial sum off by at most 2^-23 of
the sum of magnitudes, E = D 2^-23 max_j sum |q_i k_ij| scale, every weight within e^{2E}), the sums of len weights
are off by at most len 2^-24, the exponentials by 2^-20, and the output is rounded once."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_81_b200 import gdn
from gated_delta_rule_81_b200 import inputs as gin
from gpu_helpers import BF16_ULP, OUT_TOL, STATE_TOL, err_word, out_error

pytestmark = pytest.mark.gpu

KEYS = ("q", "k", "v", "z", "a", "b")


def make_tree(kind, N, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows = []
    for n in range(N):
        if kind == "chain":
            r = list(range(-1, T - 1))
        elif kind == "flat":
            r = [-1] * T
        elif kind == "none":
            r = [-2] * T
        else:  # random parents, a few absent nodes (one of them with children), padding behind
            r = [int(torch.randint(-1, t, (1,), generator=g)) if t else -1 for t in range(T)]
            if kind == "holes":
                live = max(1, T - 1 - n % 3)
                r = [p if t < live else -2 for t, p in enumerate(r)]
                if T > 4:
                    r[T // 2] = -2 if n % 2 else -9
        rows.append(r)
    return rows


def dev_tree(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ gdn_qk_norm_rope

def rope_close(y, ref):
    y = y.double().cpu().numpy()
    tol = BF16_ULP * np.abs(ref["y"]) + 2.0 ** -18 * ref["size"] + 2.0 ** -130
    bad = np.abs(y - ref["y"]) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(y - ref['y']) / tol)}"


ROPE_CASES = [  # D, R, interleaved, scaling, H_q, H_kv, tokens
    (256, 64, False, "none", 24, 4, 1), (256, 64, False, "none", 24, 4, 21), (128, 128, True, "yarn", 32, 8, 1030),
    (64, 64, False, "linear", 3, 1, 4099), (80, 16, True, "ntk", 5, 5, 7), (192, 96, False, "yarn", 7, 2, 66),
    (8, 0, False, "none", 2, 1, 5), (256, 256, False, "ntk", 1, 1, 300), (256, 256, True, "none", 33, 3, 2),
    (16, 16, False, "none", 65, 1, 3),
]


@pytest.mark.parametrize("D,R,inter,scaling,H_q,H_kv,n", ROPE_CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope(D, R, inter, scaling, H_q, H_kv, n, norm):
    g = torch.Generator().manual_seed(D + R + n)
    pad = 8
    proj = (torch.randn(n, (H_q + 2 * H_kv) * D + pad, generator=g) * 2).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in
               (proj[:, :H_q * D], proj[:, H_q * D:(H_q + H_kv) * D], proj[:, (H_q + H_kv) * D:(H_q + 2 * H_kv) * D]))
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in range(2)]
    pos = torch.randint(0, 300000, (n,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1 if n > 1 else 262143
    if n > 2:
        pos[1], pos[2] = -5, 0
    kw = dict(scaling=scaling, factor=4.0 if scaling != "none" else 1.0, original_len=4096)
    rope = gdn.make_rope(D, R, base=1e6, interleaved=inter, **kw)
    n_rows = n + 5
    rows = torch.randperm(n_rows, generator=g)[:n]
    if n > 4:
        rows[3] = -1
    k_out = torch.full((n_rows, H_kv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v_out = k_out.clone()
    err = err_word()
    before = proj.clone()
    y, _, _ = gdn.qk_norm_rope(rope, q, k, v, q_norm_w=w[0], k_norm_w=w[1], positions=pos.cuda(), rows=rows.cuda(),
                               k_out=k_out, v_out=v_out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(proj, before)
    theta, amp = oracle.tree.rope_frequencies(R, 1e6, **kw) if R else (None, 1.0)
    rope_close(y, oracle.tree.norm_rope(q.cpu(), None if w[0] is None else w[0].cpu(), pos.numpy(), R, inter, theta, amp))
    kept = rows >= 0
    ref = oracle.tree.norm_rope(k.cpu(), None if w[1] is None else w[1].cpu(), pos.numpy(), R, inter, theta, amp)
    rope_close(k_out[rows[kept].cuda()], {x: ref[x][kept.numpy()] for x in ref})
    assert torch.equal(v_out[rows[kept].cuda()], v[kept.cuda()])
    rest = torch.ones(n_rows, dtype=torch.bool)
    rest[rows[kept]] = False
    assert bool((k_out[rest.cuda()] == 7).all()) and bool((v_out[rest.cuda()] == 7).all())


@pytest.mark.parametrize("D,H_q,H_kv,n", [(256, 3, 1, 4736 + 37), (128, 5, 2, 2 * 9472 + 900), (128, 2, 1, 9472), (64, 3, 2, 18944 + 9000)])
def test_qk_norm_rope_more_tokens_than_fit_at_once(D, H_q, H_kv, n):
    """Rounds of whole tokens, then the tokens left over, split or whole: bitwise the results of small calls."""
    g = torch.Generator().manual_seed(n)
    proj = torch.randn(n, (H_q + 2 * H_kv) * D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in (proj[:, :H_q * D], proj[:, H_q * D:(H_q + H_kv) * D], proj[:, (H_q + H_kv) * D:]))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 300000, (n,), generator=g, dtype=torch.int32).cuda()
    rows = torch.randperm(n, generator=g).cuda()
    rope = gdn.make_rope(D, D // 2, base=1e6)
    outs = []
    for step in (n, 611):
        k_out, v_out = (torch.zeros(n, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        y = torch.cat([gdn.qk_norm_rope(rope, q[i:i + step], k[i:i + step], v[i:i + step], q_norm_w=w, k_norm_w=w,
                                        positions=pos[i:i + step], rows=rows[i:i + step], k_out=k_out, v_out=v_out)[0]
                       for i in range(0, n, step)])
        outs.append((y, k_out, v_out))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][2][rows], v)


def test_qk_norm_rope_in_place_parts_and_bad_rows():
    D, n = 128, 37
    g = torch.Generator().manual_seed(5)
    proj = torch.randn(n, 6 * D, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    rope = gdn.make_rope(D, 64)
    q, k = proj[:, :4 * D].unflatten(1, (4, D)), proj[:, 4 * D:].unflatten(1, (2, D))
    want_q, want_k, _ = gdn.qk_norm_rope(rope, q, k, q_norm_w=w, k_norm_w=w)  # positions 0, 1, ..
    only_q, _, _ = gdn.qk_norm_rope(rope, q, q_norm_w=w)
    _, only_k, _ = gdn.qk_norm_rope(rope, None, k, k_norm_w=w)
    assert torch.equal(only_q, want_q) and torch.equal(only_k, want_k)
    theta, amp = oracle.tree.rope_frequencies(64, 1e7)
    rope_close(want_q, oracle.tree.norm_rope(q.cpu(), w.cpu(), np.arange(n), 64, False, theta, amp))
    err = err_word()
    rows = torch.arange(n, device="cuda")
    rows[4] = n
    k_out = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda")
    gdn.qk_norm_rope(rope, q, k, q_norm_w=w, k_norm_w=w, rows=rows, k_out=k_out, err=err)
    assert int(err.item()) == 128 and bool((k_out[4] == 0).all())
    keep = torch.arange(n, device="cuda") != 4
    assert torch.equal(k_out[keep], want_k[keep])
    q2, k2, _ = gdn.qk_norm_rope(rope, q, k, q_norm_w=w, k_norm_w=w, q_out=q, k_out=k)  # both in place
    assert torch.equal(q2, want_q) and torch.equal(k2, want_k) and q2.data_ptr() == proj.data_ptr()


# ------------------------------------------------------------------ gdn_attention_tree

def attn_case(N, T, H, Hkv, D, lens, kind="holes", seed=0, gate=True, cap=None, stale=float("nan")):
    """Operands on the GPU; cache rows past each length and absent nodes hold `stale`."""
    g = torch.Generator().manual_seed(seed)
    cap = cap or max(max(lens), 1) + 3
    rows = make_tree(kind, N, T, seed)
    proj = torch.randn(N * T, (H + 2 * Hkv) * D + 8, generator=g).to(torch.bfloat16)
    q = torch.randn(N * T, H, D, generator=g).to(torch.bfloat16)
    there = torch.tensor([bool(p) for r in rows for p in oracle.tree.paths(r)])
    proj[~there] = stale
    q[~there] = stale
    kc, vc = (torch.randn(N, cap, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    for n, L in enumerate(lens):
        kc[n, L:] = stale
        vc[n, L:] = stale
    proj = proj.cuda()
    c = dict(q=q.cuda(), kc=kc.cuda(), vc=vc.cuda(), rows=rows, parent=dev_tree(rows), T=T,
             len=torch.tensor(lens, dtype=torch.int32, device="cuda"), lens=lens)
    c["g"] = proj[:, :H * D].unflatten(1, (H, D)) if gate else None
    c["kt"], c["vt"] = (proj[:, (H + i * Hkv) * D:(H + (i + 1) * Hkv) * D].unflatten(1, (Hkv, D)) for i in range(2))
    return c


def attn_run(c, **kw):
    return gdn.attention_tree(c["q"], c["kt"], c["vt"], c["kc"], c["vc"], c["len"], c["parent"], g=c["g"], **kw)


def attn_check(c, out, nodes=None, scale=None):
    ref = oracle.tree.attention_tree(c["q"].cpu(), c["kt"].cpu(), c["vt"].cpu(), c["kc"].cpu(), c["vc"].cpu(), c["lens"],
                                     c["rows"], None if c["g"] is None else c["g"].cpu(), scale)
    D = c["q"].shape[2]
    there = np.array([bool(p) for r in c["rows"] for p in oracle.tree.paths(r)])
    y = out.view(c["q"].shape).double().cpu().numpy()
    assert np.all(y[~there] == 0), "an absent node's row is not zeros"
    y, r, mass, shift = (x[there] for x in (y, ref["out"], ref["mass"], ref["shift"]))
    E = D * 2.0 ** -23 * shift
    rel = (1 + BF16_ULP + 2.0 ** -20) * np.exp(2 * E) * (1 + (max(c["lens"]) + 64) * 2.0 ** -24) - 1
    tol = (rel * mass) * (1 + BF16_ULP) + BF16_ULP * np.abs(r) + 1e-30
    bad = ~(np.abs(y - r) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(y - r) / tol)}"


ATTN_CASES = [  # N, T, H, Hkv, D, lens
    (1, 1, 24, 4, 256, [0]), (1, 1, 24, 4, 256, [1]), (1, 1, 24, 4, 256, [777]), (2, 2, 24, 4, 256, [63, 64]),
    (3, 5, 24, 4, 256, [65, 0, 1023]), (1, 21, 24, 4, 256, [300]), (2, 22, 24, 4, 256, [129, 64]),
    (1, 64, 24, 4, 256, [2049]), (4, 33, 6, 1, 256, [5, 500, 127, 128]), (5, 7, 32, 8, 128, [64, 1, 0, 333, 64]),
    (2, 64, 16, 1, 128, [100, 700]), (3, 16, 4, 4, 128, [640, 7, 65]), (2, 9, 5, 1, 128, [191, 192]),
    (37, 3, 8, 2, 256, [(i * 53) % 400 for i in range(37)]), (1, 64, 1, 1, 256, [4097]), (200, 1, 2, 2, 128, [3] * 200),
]


@pytest.mark.parametrize("N,T,H,Hkv,D,lens", ATTN_CASES)
@pytest.mark.parametrize("kind", ["holes", "chain"])
def test_attention_tree(N, T, H, Hkv, D, lens, kind):
    """Against the oracle; everything no node may see (stale rows, absent nodes) is NaN."""
    c = attn_case(N, T, H, Hkv, D, lens, kind, seed=N + T, gate=kind == "holes")
    err = err_word()
    out = attn_run(c, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(c, out)
    if kind == "chain":
        c["parent"] = None
        assert torch.equal(attn_run(c, T=T), out)
    assert torch.equal(attn_run(c), out), "a second call differs"


def test_attention_tree_scale_and_flat_tree():
    c = attn_case(2, 12, 8, 2, 128, [200, 31], "flat", seed=3)
    attn_check(c, attn_run(c, scale=0.25), scale=0.25)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attention_tree_infinities_stay_on_their_paths(value):
    """A node whose key and value are not finite reaches its descendants and no other node."""
    N, T, bad = 1, 24, 3
    c = attn_case(N, T, 24, 4, 256, [150], "holes", seed=9)
    clean = attn_run(c).view(T, 24, 256)
    for x in (c["kt"], c["vt"]):
        x[bad] = value
    out = attn_run(c).view(T, 24, 256)
    hit = torch.tensor([bad in p for p in oracle.tree.paths(c["rows"][0])], device="cuda")
    assert bool(hit.any()) and bool((~hit).any())
    assert torch.equal(out[~hit], clean[~hit])
    # the value alone: the exact result is that of the definition, element by element
    c = attn_case(N, T, 24, 4, 256, [150], "holes", seed=9)
    c["vt"][bad, :, 5] = value
    out = attn_run(c).view(T, 24, 256)
    assert torch.equal(out[~hit], clean[~hit])
    there = torch.ones(256, dtype=torch.bool, device="cuda")
    there[5] = False
    assert torch.equal(out[..., there], clean[..., there])
    got = out[hit][..., 5]
    assert bool(torch.isnan(got).all()) if value != value else bool((got == value).all())


def test_attention_tree_lowest_values_and_empty_softmax_blocks():
    """Scores at the type's lowest values in whole key blocks, and an infinite score at a masked node."""
    c = attn_case(1, 6, 4, 4, 128, [192], "chain", seed=4, gate=False)
    low = torch.finfo(torch.bfloat16).min
    c["q"].fill_(1.0)
    c["kc"][0, :128] = low / 256  # the first two blocks of keys: scores of about -1e37 and below
    c["kc"][0, 128:192] = 0.0
    out = attn_run(c)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
    attn_check(c, out)


def test_attention_tree_bad_lengths():
    c = attn_case(3, 4, 8, 2, 128, [50, 60, 70], "chain", seed=6)
    want = attn_run(c).view(3, 4, -1)
    for value in (-1, c["kc"].shape[1] + 1, 2 ** 31 - 1, -2 ** 31):
        c["len"][1] = value
        err = err_word()
        out = attn_run(c, err=err).view(3, 4, -1)
        assert int(err.item()) == 32
        assert bool((out[1] == 0).all()) and torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


def test_attention_tree_every_length_bad():
    c = attn_case(5, 3, 8, 2, 128, [10] * 5, "chain", seed=12)
    c["len"].fill_(-3)
    err = err_word()
    out = attn_run(c, err=err)
    assert int(err.item()) == 32 and bool((out == 0).all())


@pytest.mark.parametrize("N,T", [(700, 1), (1300, 2)])
def test_attention_tree_more_sequences_than_threads(N, T):
    """The work split sums several sequences per thread; some are empty, some out of range."""
    lens = [(i * 37) % 200 if i % 11 else 0 for i in range(N)]
    c = attn_case(N, T, 2, 1, 128, lens, "chain", seed=N)
    want = attn_run(c).view(N, T, -1)
    attn_check(c, want.reshape(N * T, -1))
    bad = torch.tensor([i for i in range(N) if i % 97 == 5], device="cuda")
    c["len"][bad] = -1
    err = err_word()
    out = attn_run(c, err=err).view(N, T, -1)
    assert int(err.item()) == 32 and bool((out[bad] == 0).all())
    good = torch.ones(N, dtype=torch.bool, device="cuda")
    good[bad] = False
    c["len"][bad] = torch.tensor([lens[int(i)] for i in bad], dtype=torch.int32, device="cuda")
    # (another split of the work: the same sums in another order)
    assert float((out[good].float() - want[good].float()).abs().max()) <= 4 * BF16_ULP * float(want.float().abs().max())


def test_attention_tree_two_streams_and_rows_beside_the_output():
    """Two calls at once on two streams, each with its own workspace and an output inside a larger buffer whose other
    rows stay as they are."""
    cases = [attn_case(2, 9, 24, 4, 256, [1500, 800], "holes", seed=40), attn_case(3, 20, 8, 2, 128, [700, 64, 2100], "holes", seed=41)]
    wants = [attn_run(c) for c in cases]
    bufs = [torch.full((w.shape[0] + 2, w.shape[1]), 5.0, dtype=torch.bfloat16, device="cuda") for w in wants]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, b, s in zip(cases, bufs, streams):
            with torch.cuda.stream(s):
                attn_run(c, out=b[1:-1])
    torch.cuda.synchronize()
    for w, b in zip(wants, bufs):
        assert torch.equal(b[1:-1], w) and bool((b[0] == 5).all()) and bool((b[-1] == 5).all())


@pytest.mark.parametrize("D,H,Hkv", [(256, 24, 4), (128, 32, 8)])
def test_attention_tree_repeats_bitwise_under_load(D, H, Hkv):
    """Many ragged contexts whose tiles stream from memory as fast as it gives them: every repetition gives the same bits,
    whatever the order in which copies land."""
    N, T, cap = 64, 16, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    kc, vc = rnd(N, cap, Hkv, D), rnd(N, cap, Hkv, D)
    q, kt, vt, gate = rnd(N * T, H * D), rnd(N * T, Hkv * D), rnd(N * T, Hkv * D), rnd(N * T, H * D)
    lens = torch.tensor([300 + (cap - 300) * ((i * 7) % N) // (N - 1) for i in range(N)], dtype=torch.int32, device="cuda")
    parent = dev_tree(make_tree("holes", N, T, 3))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    want = None
    for rep in range(60):
        flush.fill_(rep)
        out = gdn.attention_tree(q.view(N * T, H, D), kt.view(N * T, Hkv, D), vt.view(N * T, Hkv, D), kc, vc, lens, parent,
                                 g=gate.view(N * T, H, D))
        want = out if want is None else want
        assert torch.equal(out, want), rep


def test_tree_bad_parents_are_absent_and_reported():
    c = attn_case(1, 5, 8, 2, 128, [40], "chain", seed=7)
    want = attn_run(c).view(5, -1)
    c["parent"][0, 3] = 3  # itself: no earlier node
    err = err_word()
    out = attn_run(c, err=err).view(5, -1)
    assert int(err.item()) == 128
    assert torch.equal(out[:3], want[:3]) and bool((out[3:] == 0).all())
    c["parent"][0, 3] = 2 ** 31 - 1
    assert torch.equal(attn_run(c).view(5, -1), out)


def test_attention_tree_offsets_past_32_bits():
    """Caches of more than 2^31 elements each: the last sequence's rows lie beyond 32-bit offsets."""
    N, cap, H, Hkv, D, T = 9, 262144, 24, 4, 256, 2
    kc, vc = (torch.zeros(N, cap, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    g = torch.Generator().manual_seed(1)
    L = 500
    tail = [torch.randn(L, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    kc[N - 1, :L], vc[N - 1, :L] = tail[0].cuda(), tail[1].cuda()
    lens = [0] * (N - 1) + [L]
    c = attn_case(N, T, H, Hkv, D, lens, "chain", seed=2, cap=L)
    small = attn_run(c | {"kc": kc[:, :L].contiguous(), "vc": vc[:, :L].contiguous()})
    out = attn_run(c | {"kc": kc, "vc": vc})
    assert torch.equal(out, small)
    attn_check(c | {"kc": kc[:, :L].cpu(), "vc": vc[:, :L].cpu()}, out)


def test_attention_tree_graph_stream_and_shared_pool():
    """Captured into a graph and replayed on other contents, on a stream of its own."""
    c = attn_case(3, 8, 24, 4, 256, [333, 70, 900], "holes", seed=8)
    d = attn_case(3, 8, 24, 4, 256, [901, 3, 64], "holes", seed=18, cap=c["kc"].shape[1])
    want_c, want_d = attn_run(c), attn_run(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want_c)
    with torch.cuda.stream(s):
        attn_run(c, out=out)  # warm-up
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            attn_run(c, out=out)
        for name, want in ((c, want_c), (d, want_d), (c, want_c)):
            if name is d:
                saved = {k: c[k].clone() for k in ("q", "kc", "vc", "len", "parent", "g", "kt", "vt")}
                for k in saved:
                    c[k].copy_(d[k])
            graph.replay()
            s.synchronize()
            assert torch.equal(out, want)
            if name is d:
                for k in saved:
                    c[k].copy_(saved[k])


# ------------------------------------------------------------------ gdn_decode_tree and its commit

def delta_case(N, T, H_k, H_v, kind="holes", seed=0, slots=None, a_mean=0.0, bad=float("nan")):
    """Pools with `slots` slots, sequence n in a slot of its own; absent nodes' inputs are `bad`."""
    slots = slots or N
    g = torch.Generator().manual_seed(seed)
    rows = make_tree(kind, N, T, seed)
    inp = gin.token_inputs(N * T, H_k, H_v, seed=seed, a_mean=a_mean)
    there = torch.tensor([bool(p) for r in rows for p in oracle.tree.paths(r)])
    for k in KEYS:
        inp[k][~there] = bad
    inp.update(gin.weights(H_k, H_v, seed=seed))
    inp["scale"] = 0.7
    slot = torch.randperm(slots, generator=g)[:N].to(torch.int32)
    state = gin.recurrent_state(slots, H_v, seed=seed + 1)
    conv = gin.conv_state(slots, H_k, H_v, seed=seed + 2)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}
    s = gdn.make_inputs(*(dev[k] for k in ("q", "k", "v", "a", "b", "z")), dev["conv_w"], dev["A_log"], dev["norm_w"],
                        scale=inp["scale"])
    return dict(inp=inp, dev=dev, s=s, rows=rows, parent=dev_tree(rows), slot=slot, N=N, T=T, there=there,
                state=state, conv=conv, d_state=state.cuda(), d_conv=conv.cuda(), d_slot=slot.cuda())


def delta_ref(c):
    sl = c["slot"].long()
    return oracle.tree.mixer_tree({k: torch.nan_to_num(v) if k in KEYS else v for k, v in c["inp"].items()}, c["rows"],
                                  c["state"][sl], c["conv"][sl])


DELTA_CASES = [  # N, T, H_k, H_v
    (1, 1, 2, 6), (3, 2, 2, 6), (1, 7, 2, 6), (2, 8, 1, 8), (1, 9, 3, 3), (2, 13, 2, 4), (1, 16, 16, 48), (3, 17, 1, 3),
    (1, 31, 2, 6), (1, 33, 2, 2), (1, 48, 1, 5), (2, 61, 2, 6), (1, 64, 1, 8), (90, 3, 2, 4),
]


@pytest.mark.parametrize("N,T,H_k,H_v", DELTA_CASES)
@pytest.mark.parametrize("kind", ["holes", "chain"])
def test_decode_tree(N, T, H_k, H_v, kind):
    c = delta_case(N, T, H_k, H_v, kind, seed=N + T + H_v, slots=N + 2, a_mean=0.0 if kind == "holes" else -4.0)
    err = err_word()
    before = c["d_state"].clone(), c["d_conv"].clone()
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"], err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(c["d_state"], before[0]) and torch.equal(c["d_conv"], before[1])
    ref = delta_ref(c)
    assert bool((out[~c["there"].cuda()] == 0).all())
    t = c["there"].numpy()
    e = out_error(out[c["there"].cuda()], ref["out"][t])
    print(f"[parity] decode_tree N={N} T={T} H={H_k}/{H_v} {kind}: out_err={e:.3e}")
    assert e <= OUT_TOL
    again = gdn.decode_tree(c["s"], N, T, c["parent"] if kind == "holes" else None, c["d_state"], c["d_conv"],
                            state_slot=c["d_slot"])
    assert torch.equal(again, out)


@pytest.mark.parametrize("T,H_v", [(5, 3), (16, 3), (16, 8), (32, 3), (29, 8), (40, 3), (64, 2), (33, 8)])
def test_decode_tree_large_batch(T, H_v):
    """Many sequences: one CTA takes all the value heads of a key head in turn.  Bitwise the results of a few
    sequences, whose value heads have a CTA each, and within the bound of the oracle."""
    N, H_k = 150, 1
    c = delta_case(N, T, H_k, H_v, "holes", seed=77 + T)
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"]).view(N, T, H_v, 128)
    seqs = list(range(0, N, 29))
    rows = torch.tensor([n * T + t for n in seqs for t in range(T)], device="cuda")
    few = {k: c["dev"][k][rows].contiguous() for k in KEYS}
    s = gdn.make_inputs(*(few[k] for k in ("q", "k", "v", "a", "b", "z")), c["dev"]["conv_w"], c["dev"]["A_log"], c["dev"]["norm_w"],
                        scale=c["inp"]["scale"])
    alone = gdn.decode_tree(s, len(seqs), T, c["parent"][seqs].contiguous(), c["d_state"], c["d_conv"],
                            state_slot=c["d_slot"][seqs].contiguous()).view(len(seqs), T, H_v, 128)
    assert torch.equal(alone, out[seqs])
    sub = dict(c, rows=[c["rows"][n] for n in seqs], slot=c["slot"][seqs],
               inp={k: v[rows.cpu()] if k in KEYS else v for k, v in c["inp"].items()})
    there = c["there"].view(N, T)[seqs].reshape(-1)
    ref = delta_ref(sub)["out"][there.numpy()]
    assert out_error(alone.reshape(-1, H_v, 128)[there.cuda()], ref) <= OUT_TOL


@pytest.mark.parametrize("T,H_v", [(1, 2), (8, 8), (7, 5), (4, 3), (64, 8), (61, 4), (37, 3), (33, 6)])
def test_decode_tree_large_batch_with_bad_slots_and_nodes(T, H_v):
    """Many sequences, several value heads per CTA: slots that are shared or out of range, a node whose key is not finite and bad
    parents, each without effect on the other sequences, which keep bitwise the results that they have alone."""
    N, H_k = 150, 1
    c = delta_case(N, T, H_k, H_v, "holes", seed=177 + T)
    slot = c["slot"].clone()
    slot[3], slot[70], slot[149], slot[20] = N, -1, 2 ** 31 - 1, slot[21]
    seq = 40
    bad = int(c["there"].view(N, T)[seq].nonzero()[0])
    c["dev"]["k"][seq * T + bad] = float("inf")
    parent = c["parent"].clone()
    parent[50, T - 1] = T + 5
    err = err_word()
    out = gdn.decode_tree(c["s"], N, T, parent, c["d_state"], c["d_conv"], state_slot=slot.cuda(), err=err).view(N, T, H_v, 128)
    torch.cuda.synchronize()
    assert int(err.item()) == 8 | 128
    assert bool((out[[3, 70, 149]] == 0).all())
    assert bool((out[50, T - 1] == 0).all())
    hit = torch.tensor([bad in p for p in oracle.tree.paths(c["rows"][seq])], device="cuda")
    assert bool(torch.isnan(out[seq][hit]).all()) and not bool(torch.isnan(out[seq][~hit]).any())
    for n in (0, 20, 21, seq, 50, 101, 148):
        rows = torch.arange(n * T, (n + 1) * T, device="cuda")
        one = {k: c["dev"][k][rows].contiguous() for k in KEYS}
        s = gdn.make_inputs(*(one[k] for k in ("q", "k", "v", "a", "b", "z")), c["dev"]["conv_w"], c["dev"]["A_log"],
                            c["dev"]["norm_w"], scale=c["inp"]["scale"])
        alone = gdn.decode_tree(s, 1, T, parent[n:n + 1].contiguous(), c["d_state"], c["d_conv"], state_slot=slot[n:n + 1].cuda())
        assert torch.equal(alone.view(T, H_v, 128).view(torch.int16), out[n].view(torch.int16)), n


@pytest.mark.parametrize("T,N", [(5, 90), (13, 2), (30, 2), (40, 2), (64, 90)])
def test_decode_tree_pools_and_rows_aligned_to_16_bytes_only(T, N):
    """A state pool, conv pool and rows that begin 16 bytes into their buffers: the results of aligned ones, bitwise."""
    H_k, H_v = 2, 6
    c = delta_case(N, T, H_k, H_v, "holes", seed=T)
    want = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])

    def moved(x):
        step = 16 // x.element_size()
        buf = torch.zeros(x.numel() + 2 * step, dtype=x.dtype, device="cuda")
        y = buf[step:step + x.numel()].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        return y

    d = c["dev"]
    m = {k: moved(d[k]) for k in ("q", "k", "v", "z", "conv_w")}  # (kept: the descriptor holds addresses)
    s = gdn.make_inputs(m["q"], m["k"], m["v"], d["a"], d["b"], m["z"], m["conv_w"], d["A_log"], d["norm_w"], scale=c["inp"]["scale"])
    state, conv, out = moved(c["d_state"]), moved(c["d_conv"]), moved(torch.zeros_like(want))
    gdn.decode_tree(s, N, T, c["parent"], state, conv, state_slot=c["d_slot"], out=out)
    assert torch.equal(out, want)


def test_decode_tree_and_commit_past_32_bit_offsets():
    """A pool of more than 2^31 state elements: the sequence's slot is the last."""
    T, H_k, H_v, slots = 9, 16, 48, 2800
    c = delta_case(1, T, H_k, H_v, "chain", seed=3)
    state = torch.zeros(slots, H_v, 128, 128, device="cuda")
    assert state.numel() > 2 ** 31
    conv = torch.zeros(slots, 3, (2 * H_k + H_v) * 128, dtype=torch.bfloat16, device="cuda")
    state[-1], conv[-1] = c["d_state"][0], c["d_conv"][0]
    slot = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    acc = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    want = gdn.decode_tree(c["s"], 1, T, c["parent"], c["d_state"], c["d_conv"])
    assert torch.equal(gdn.decode_tree(c["s"], 1, T, c["parent"], state, conv, state_slot=slot), want)
    S, C = c["d_state"].clone(), c["d_conv"].clone()
    gdn.decode_tree_commit(c["s"], 1, T, c["parent"], acc, S, C)
    gdn.decode_tree_commit(c["s"], 1, T, c["parent"], acc, state, conv, state_slot=slot)
    assert torch.equal(state[-1], S[0]) and torch.equal(conv[-1], C[0])
    assert not bool(state[:-1].any()) and not bool(conv[:-1].any())


@pytest.mark.parametrize("key", ["q", "k", "v", "a", "b", "z"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [7, 16, 40])
def test_decode_tree_infinities_stay_on_their_paths(key, value, T):
    """A node whose input is not finite reaches its descendants (through its key, value or gates) or itself alone
    (its query and output gate), and no other node."""
    N, H_k, H_v, bad = 1, 2, 6, 2
    c = delta_case(N, T, H_k, H_v, "holes", seed=31 + T)
    clean = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])
    c["dev"][key][bad] = value
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])
    hit = torch.tensor([bad in p for p in oracle.tree.paths(c["rows"][0])], device="cuda")
    assert bool(hit.any()) and bool((~hit).any())
    assert torch.equal(out[~hit], clean[~hit])
    if value != value and key != "z":
        assert bool(torch.isnan(out[bad]).all())
        if key in ("k", "v", "a", "b"):
            assert bool(torch.isnan(out[hit]).all())


def test_decode_tree_shared_and_bad_slots():
    N, T, H_k, H_v = 4, 6, 2, 6
    c = delta_case(N, T, H_k, H_v, "chain", seed=5, slots=6)
    slot = torch.tensor([2, 2, 7, -1], dtype=torch.int32)
    err = err_word()
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=slot.cuda(), err=err).view(N, T, H_v, 128)
    assert int(err.item()) == 8
    assert bool((out[2:] == 0).all())
    c["slot"] = torch.tensor([2, 2, 0, 0])
    ref = delta_ref(c)["out"].reshape(N, T, H_v, 128)
    assert out_error(out[:2].reshape(-1, H_v, 128), ref[:2].reshape(-1, H_v, 128)) <= OUT_TOL


COMMIT_CASES = [(1, 1, 2, 6), (3, 5, 2, 6), (2, 16, 16, 48), (4, 33, 1, 8), (100, 4, 2, 4), (2, 64, 1, 3), (70, 20, 3, 6)]


@pytest.mark.parametrize("N,T,H_k,H_v", COMMIT_CASES)
@pytest.mark.parametrize("kind", ["holes", "chain"])
@pytest.mark.parametrize("in_place", [True, False])
def test_decode_tree_commit_is_bitwise_decoding_the_path(N, T, H_k, H_v, kind, in_place):
    c = delta_case(N, T, H_k, H_v, kind, seed=N + T, slots=N + 2)
    ps = [oracle.tree.paths(r) for r in c["rows"]]
    accepted = []
    for n in range(N):
        live = [t for t in range(T) if ps[n][t]]
        accepted.append(-1 if n % 5 == 4 else live[(n * 3) % len(live)] if n else live[-1])
    acc = torch.tensor(accepted, dtype=torch.int32, device="cuda")
    want_S, want_C = c["d_state"].clone(), c["d_conv"].clone()
    # the sequences' paths token by token through decode_step (one sequence at a time, in its slot)
    for n in range(N if N <= 4 else 6):
        path = ps[n][accepted[n]] if accepted[n] >= 0 else []
        slot = c["d_slot"][n:n + 1].contiguous()
        for t in path:
            row = n * T + t
            one = {k: c["dev"][k][row:row + 1].contiguous() for k in KEYS}
            s = gdn.make_inputs(*(one[k] for k in ("q", "k", "v", "a", "b", "z")), c["dev"]["conv_w"], c["dev"]["A_log"],
                                c["dev"]["norm_w"], scale=c["inp"]["scale"])
            gdn.decode_multi(s, 1, 1, want_S, want_C, state_slot=slot)
    S, C = c["d_state"].clone(), c["d_conv"].clone()
    S2, C2 = (S, C) if in_place else (torch.full_like(S, 3.0), torch.full_like(C, 3.0))
    err = err_word()
    gdn.decode_tree_commit(c["s"], N, T, c["parent"], acc, S, C, state_slot=c["d_slot"], state_out=S2, conv_out=C2, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    seqs = c["slot"].long()[:N if N <= 4 else 6].cuda()
    assert torch.equal(S2[seqs], want_S[seqs]) and torch.equal(C2[seqs], want_C[seqs])
    others = torch.ones(N + 2, dtype=torch.bool)
    others[c["slot"].long()] = False
    if in_place:
        assert torch.equal(S2[others.cuda()], c["d_state"][others.cuda()])
    else:
        assert torch.equal(S, c["d_state"]) and torch.equal(C, c["d_conv"])
        assert bool((S2[others.cuda()] == 3).all()) and bool((C2[others.cuda()] == 3).all())
    ref = delta_ref(c)
    for n in range(N):
        got = S2[int(c["slot"][n])].double().cpu().numpy()
        tok = n * T + accepted[n]
        r = ref["state"][tok] if accepted[n] >= 0 else c["state"][int(c["slot"][n])].double().numpy()
        assert np.linalg.norm(got - r) <= STATE_TOL * np.linalg.norm(r)
        if accepted[n] >= 0:
            np.testing.assert_array_equal(C2[int(c["slot"][n])].float().cpu().numpy(), ref["conv"][tok])


def test_decode_tree_commit_bad_entries():
    N, T, H_k, H_v = 4, 6, 2, 6
    c = delta_case(N, T, H_k, H_v, "chain", seed=15)
    c["parent"][1, 3:] = -2
    acc = torch.tensor([6, 4, -7, 2], dtype=torch.int32, device="cuda")  # past the tree, absent, negative; one good
    S, C = c["d_state"].clone(), c["d_conv"].clone()
    err = err_word()
    gdn.decode_tree_commit(c["s"], N, T, c["parent"], acc, S, C, state_slot=c["d_slot"], err=err)
    assert int(err.item()) == 128
    same = c["d_slot"][:3].long()
    assert torch.equal(S[same], c["d_state"][same]) and torch.equal(C[same], c["d_conv"][same])
    assert not torch.equal(S[c["d_slot"][3].long()], c["d_state"][c["d_slot"][3].long()])
    err.zero_()
    bad = torch.tensor([0, 9, -1, 1], dtype=torch.int32, device="cuda")
    gdn.decode_tree_commit(c["s"], N, T, c["parent"], torch.full_like(acc, -1), S, C, state_slot=bad, err=err)
    assert int(err.item()) == 8


def test_decode_tree_graph_replay():
    """Verification and commit captured together, replayed twice: the second replay continues from the first's state."""
    N, T, H_k, H_v = 2, 9, 2, 6
    c = delta_case(N, T, H_k, H_v, "holes", seed=21)
    acc = torch.tensor([t[-1] if t else -1 for t in ([i for i in range(T) if p[i]] for p in
                                                     (oracle.tree.paths(r) for r in c["rows"]))], dtype=torch.int32, device="cuda")
    S, C = c["d_state"].clone(), c["d_conv"].clone()
    wants = []
    for _ in range(2):
        wants.append(gdn.decode_tree(c["s"], N, T, c["parent"], S, C, state_slot=c["d_slot"]))
        gdn.decode_tree_commit(c["s"], N, T, c["parent"], acc, S, C, state_slot=c["d_slot"])
    S2, C2 = c["d_state"].clone(), c["d_conv"].clone()
    out = torch.empty_like(wants[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            gdn.decode_tree(c["s"], N, T, c["parent"], S2, C2, state_slot=c["d_slot"], out=out)
            gdn.decode_tree_commit(c["s"], N, T, c["parent"], acc, S2, C2, state_slot=c["d_slot"])
        for want in wants:
            graph.replay()
            st.synchronize()
            assert torch.equal(out, want)
    assert torch.equal(S2, S) and torch.equal(C2, C)


# ------------------------------------------------------------------ gdn_attn_tree_commit

@pytest.mark.parametrize("N,T,Hkv,D", [(1, 1, 4, 256), (5, 31, 8, 128), (3, 64, 1, 128), (130, 9, 2, 256)])
@pytest.mark.parametrize("kind", ["holes", "chain"])
def test_attn_tree_commit(N, T, Hkv, D, kind):
    g = torch.Generator().manual_seed(N * T)
    rows = make_tree(kind, N, T, seed=T)
    cap = T + 20
    proj = torch.randn(N * T, 2 * Hkv * D + 16, generator=g).to(torch.bfloat16).cuda()
    kt, vt = proj[:, :Hkv * D].unflatten(1, (Hkv, D)), proj[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D))
    kc, vc = (torch.randn(N, cap, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ps = [oracle.tree.paths(r) for r in rows]
    acc, lens, want, fits = [], [], [], True
    wk, wv = kc.clone(), vc.clone()
    for n in range(N):
        live = [t for t in range(T) if ps[n][t]]
        acc.append(-1 if n % 4 == 3 else live[-1 - (n % len(live))])
        path = ps[n][acc[n]] if acc[n] >= 0 else []
        lens.append([0, cap - len(path), 11, cap][n % 4] if n % 7 != 6 else cap - len(path) + 1)
        room = lens[n] <= cap and lens[n] + len(path) <= cap
        fits &= room or not path
        if room:
            for i, t in enumerate(path):
                wk[n, lens[n] + i], wv[n, lens[n] + i] = kt[n * T + t], vt[n * T + t]
        want.append(lens[n] + len(path) if room else lens[n])
    ok_len = all(0 <= x <= cap for x in lens)
    d_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(d_len)
    err = err_word()
    a = torch.tensor(acc, dtype=torch.int32, device="cuda")
    kc0, vc0 = kc.clone(), vc.clone()
    gdn.attn_tree_commit(kt, vt, T, dev_tree(rows), a, kc, vc, d_len, cache_len_out=new, err=err)
    assert int(err.item()) == (0 if fits else 16) | (0 if ok_len else 32)
    assert new.tolist() == want and d_len.tolist() == lens
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    gdn.attn_tree_commit(kt, vt, T, dev_tree(rows), a, kc0, vc0, d_len)  # the lengths in place
    assert d_len.tolist() == want and torch.equal(kc0, wk) and torch.equal(vc0, wv)


# ------------------------------------------------------------------ the layers, together

def test_hybrid_layers_verify_and_commit_a_tree_as_token_by_token_decoding_does():
    """A delta-rule layer and an attention layer: prompt, a tree of drafts through both layers, the accepted
    path committed, one more step; against decoding the same tokens one at a time."""
    g = torch.Generator().manual_seed(11)
    hidden, H_k, H_v, N, P, T = 128, 2, 6, 2, 70, 11
    n_in = int(gdn.load().gdn_layer_n_in(H_k, H_v))

    def mat(r, c):
        return (torch.randn(r, c, generator=g) * c ** -0.5).to(torch.bfloat16).cuda()

    conv_w = (torch.randn((2 * H_k + H_v) * 128, 4, generator=g) * 0.5).to(torch.bfloat16).cuda()
    A_log = (torch.rand(H_v, generator=g) * 2).cuda()
    ones = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    w = [mat(n_in, hidden), mat(hidden, H_v * 128), mat(gdn.ATTN_N_IN, hidden), mat(hidden, 24 * 256)]
    L1 = gdn.make_layer(w[0], w[1], conv_w, A_log, ones[:128], H_k, H_v)
    L2 = gdn.make_attn_layer(w[2], w[3], ones, ones)
    prompt = torch.randn(N * P, hidden, generator=g).to(torch.bfloat16).cuda()
    h, S, C = gdn.layer_prefill(L1, N, P, prompt)
    cap = P + 16
    _, kc, vc = gdn.attn_layer_prefill(L2, N, P, h, cache_cap=cap)
    lens = torch.full((N,), P, dtype=torch.int32, device="cuda")
    rows = make_tree("holes", N, T, seed=4)
    parent = dev_tree(rows)
    x = torch.randn(N * T, hidden, generator=g).to(torch.bfloat16).cuda()
    ps = [oracle.tree.paths(r) for r in rows]
    last = [max((t for t in range(T) if ps[n][t]), key=lambda t: len(ps[n][t])) for n in range(N)]
    acc = torch.tensor(last, dtype=torch.int32, device="cuda")
    # reference: each path token by token
    ref1, ref2 = {}, {}
    for n in range(N):
        for t in range(T):
            if not ps[n][t]:
                continue
            s1, c1 = S[n:n + 1].clone(), C[n:n + 1].clone()
            k1, v1, l1 = kc[n:n + 1].clone(), vc[n:n + 1].clone(), lens[n:n + 1].clone()
            for j in ps[n][t]:
                y1 = gdn.layer_decode(L1, 1, 1, x[n * T + j:n * T + j + 1], s1, c1)
                y2 = gdn.attn_layer_decode_step(L2, y1, k1, v1, l1)
            ref1[n, t], ref2[n, t] = y1, y2
            if t == last[n]:
                ref1[n, "S"], ref1[n, "C"], ref2[n, "k"], ref2[n, "v"], ref2[n, "l"] = s1, c1, k1, v1, l1
    err = err_word()
    ws1, ws2 = gdn.layer_tree_workspace(L1, N, T, "cuda"), gdn.attn_layer_tree_workspace(N, T, "cuda")
    y1 = gdn.layer_decode_tree(L1, N, T, parent, x, S, C, ws1, err=err)
    y2 = gdn.attn_layer_decode_tree(L2, N, T, parent, y1, kc, vc, lens, ws2, err=err)
    assert lens.tolist() == [P] * N
    for n in range(N):
        for t in range(T):
            if not ps[n][t]:
                assert bool((y1[n * T + t] == 0).all())
                continue
            for got, want in ((y1[n * T + t], ref1[n, t][0]), (y2[n * T + t], ref2[n, t][0])):
                d = (got.float() - want.float()).abs()
                # both sides round to bf16 at the projection, the mixer's or attention's output and y: the mixer within
                # OUT_TOL rms, each rounding one bf16 step of the rms of its sum (bounded by that of y, with K terms random)
                assert float(d.max()) <= 4 * (OUT_TOL + BF16_ULP) * float(want.float().square().mean().sqrt()) * 3
    gdn.layer_tree_commit(L1, N, T, parent, acc, S, C, ws1, err=err)
    gdn.attn_layer_tree_commit(N, T, parent, acc, kc, vc, lens, ws2, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for n in range(N):
        depth = len(ps[n][last[n]])
        assert int(lens[n]) == P + depth == int(ref2[n, "l"][0])
        assert float((S[n] - ref1[n, "S"][0]).norm()) <= STATE_TOL * float(S[n].norm())
        assert float((kc[n, :P + depth].float() - ref2[n, "k"][0, :P + depth].float()).abs().max()) <= 0.05
        assert torch.equal(kc[n, :P], ref2[n, "k"][0, :P]) and torch.equal(vc[n, :P], ref2[n, "v"][0, :P])
    # and on from there, one token each
    nxt = torch.randn(N, hidden, generator=g).to(torch.bfloat16).cuda()
    z1 = gdn.layer_decode(L1, N, 1, nxt, S, C)
    z2 = gdn.attn_layer_decode_step(L2, z1, kc, vc, lens)
    assert bool(torch.isfinite(z2).all()) and lens.tolist() == [P + len(ps[n][last[n]]) + 1 for n in range(N)]


def test_attn_layer_tree_keys_match_decode_bitwise_positions():
    """A chain of one node is the decode step: the same key row, value row and nearly the same output."""
    g = torch.Generator().manual_seed(2)
    hidden, N, cap = 64, 3, 40
    w_in = (torch.randn(gdn.ATTN_N_IN, hidden, generator=g) * 0.125).to(torch.bfloat16).cuda()
    w_out = (torch.randn(hidden, 24 * 256, generator=g) * 0.0128).to(torch.bfloat16).cuda()
    nw = (1 + 0.1 * torch.randn(256, generator=g)).to(torch.bfloat16).cuda()
    L = gdn.make_attn_layer(w_in, w_out, nw, nw)
    kc, vc = (torch.randn(N, cap, 4, 256, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    lens = torch.tensor([0, 17, 39], dtype=torch.int32, device="cuda")
    x = torch.randn(N, hidden, generator=g).to(torch.bfloat16).cuda()
    k1, v1, l1 = kc.clone(), vc.clone(), lens.clone()
    want = gdn.attn_layer_decode_step(L, x, k1, v1, l1)
    ws = gdn.attn_layer_tree_workspace(N, 1, "cuda")
    y = gdn.attn_layer_decode_tree(L, N, 1, None, x, kc, vc, lens, ws)
    gdn.attn_layer_tree_commit(N, 1, None, torch.zeros(N, dtype=torch.int32, device="cuda"), kc, vc, lens, ws)
    torch.cuda.synchronize()
    assert torch.equal(lens, l1) and torch.equal(vc, v1)
    # the rotation of the two kernels differs by fp32 rounding only: at most one bf16 step
    assert bool(((kc.float() - k1.float()).abs() <= 2 * BF16_ULP * k1.float().abs() + 1e-6).all())
    assert float((y.float() - want.float()).abs().max()) <= 0.05 * float(want.float().abs().max())


def test_second_device_is_refused_for_mixed_tensors():
    """Tensors that do not lie on one device are refused before any launch."""
    c = attn_case(1, 2, 8, 2, 128, [9], "chain")
    with pytest.raises(ValueError):
        gdn.attention_tree(c["q"], c["kt"], c["vt"], c["kc"], c["vc"], c["len"].cpu(), c["parent"])
    with pytest.raises((ValueError, TypeError)):
        gdn.qk_norm_rope(gdn.make_rope(128), c["q"].cpu(), c["kt"])
    assert ctypes.sizeof(gdn.GdnRope) == 5 * 4 + 4 + 128 * 8
